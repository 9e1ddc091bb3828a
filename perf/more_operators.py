"""Prompts over the paged 8-bit cache, operator by operator: what a server runs for a step of new tokens, and a trainer before attention.

  rope    rotary positions of queries and keys, and their gradient (fa_rope, fa_rope_bwd)
  append  new keys, rotated on the way, and values rounded into the cache's pages; the step's queries rotated beside (fa_kv_append_rope)
  chunk   attention of a chunk of new tokens a sequence over the cache (fa_fwd_paged_chunk)

A rotation turns the pair (x1, x2) of a head's elements by the angle position * frequency; phases [rot / 2] hold each pair's frequency as whole
turns a position, in units of 2^-64 of a turn, so that position * phase modulo 2^64 is the angle.  Pairs are neighbours (interleaved) or half of the
rotated part apart; elements behind the rotated part stay as they are; an amplitude (long contexts) multiplies the rotated ones.

A serving case gives a batch of B sequences with `cached` tokens in the cache and `new` tokens in this step; their lengths follow from the case
alone, the values from the seed. Each operator is here in its plain form, in elementary torch operations.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCRATCH = 64 << 20  # the one scratch buffer that a serving program keeps for its attention calls
ONE_CALL = 1.2e12   # operations of the largest listed case


# ------------------------------------------------------------------ cases
def listed():
    return [
        # queries and keys of one decode step, as views of a fused projection: all latency
        dict(name="rope_decode_b64", op="rope", form="packed", T=64, lo=100, hi=4000, Hq=32, Hk=8, D=128, rot=128, inter=False, yarn=0, mix=1),
        # a training batch: the fused projection [B, S, heads, D] becomes the [B, H, S, D] that attention takes
        dict(name="rope_train_b4_s4096", op="rope", form="train", B=4, S=4096, Hq=16, Hk=16, D=128, rot=128, inter=False, yarn=0, mix=2),
        # its gradient at odd lengths, back into the fused layout: neighbouring pairs, half of the small head rotated
        dict(name="rope_grad_b16_s1000_d64", op="rope", form="grad", B=16, S=1000, Hq=32, Hk=32, D=64, rot=32, inter=True, yarn=0, mix=3),
        # a long prompt at far positions with stretched frequencies
        dict(name="rope_far_16384", op="rope", form="packed", T=16384, lo=100000, hi=500000, Hq=32, Hk=8, D=128, rot=128, inter=False, yarn=16, mix=4),
        # one new token for each of 64 chats: rotated and appended, the queries rotated beside
        dict(name="append_decode_b64", op="append", B=64, lo=100, hi=4000, nlo=1, nhi=1, page=64, Hkv=8, G=4, D=128, rot=128, inter=False, yarn=0, pad=0, zero=0, mix=5),
        # a long prompt goes into the cache at once, out of a fused projection
        dict(name="append_prompt_16384", op="append", B=1, lo=0, hi=0, nlo=16384, nhi=16384, page=64, Hkv=8, G=4, D=128, rot=128, inter=False, yarn=0, pad=0, zero=0, mix=6),
        # ragged prompts behind cached prefixes, the small head dimension, small pages, neighbouring pairs, part of the head; keys and values alone
        dict(name="append_ragged_d64_p16", op="append", B=16, lo=1, hi=1000, nlo=30, nhi=1000, page=16, Hkv=32, G=0, D=64, rot=32, inter=True, yarn=8, pad=7, zero=1, mix=7),
        # a few short follow-up messages, the small head dimension, no shared heads: latency
        dict(name="chunk_short_b4_d64", op="chunk", B=4, lo=100, hi=1000, nlo=5, nhi=40, page=64, Hkv=32, G=1, D=64, pad=0, zero=0, mix=8),
        # whole prompts, nothing cached before them
        dict(name="chunk_prompt_b4_4096", op="chunk", B=4, lo=0, hi=0, nlo=4096, nhi=4096, page=64, Hkv=16, G=1, D=128, pad=0, zero=0, mix=9),
        # one chunk of a long prompt, four query heads for each key/value head
        dict(name="chunk_512_after_16384", op="chunk", B=1, lo=16384, hi=16384, nlo=512, nhi=512, page=64, Hkv=8, G=4, D=128, pad=0, zero=0, mix=10),
        # a mixed step: chats with one new token beside chunks of prompts, ragged, small pages, an empty slot
        dict(name="chunk_mixed_b32_p16", op="chunk", B=32, lo=50, hi=8000, nlo=1, nhi=1024, page=16, Hkv=8, G=8, D=128, pad=3, zero=1, mix=11),
        # a later chunk of a very long prompt
        dict(name="chunk_1024_after_65536", op="chunk", B=1, lo=65536, hi=65536, nlo=1024, nhi=1024, page=128, Hkv=8, G=4, D=128, pad=0, zero=0, mix=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk"])
    D = rng.choice([64, 128])
    c = dict(op=op, D=D, mix=rng.randrange(1 << 20))
    turn = dict(rot=16 * rng.randint(1, D // 16) if rng.random() < 0.5 else D, inter=rng.choice([False, True]), yarn=rng.choice([0, 0, 4, 32]))
    if op == "rope":
        form = rng.choice(["packed", "train", "grad"])
        Hq = rng.choice([1, 4, 8, 16, 32, 40])
        Hk = rng.choice([h for h in (1, 2, 4, 8, 16, 32, 40) if Hq % h == 0])
        room = 16384 * 40 * 128 // ((Hq + Hk) * D)  # tokens of the largest listed work
        c.update(form=form, Hq=Hq, Hk=Hk, **turn)
        if form == "packed":
            hi = _log_int(rng, 2, 1 << 20)
            c.update(T=_log_int(rng, 1, min(65536, room)), lo=rng.choice([0, hi // 2]), hi=hi)
        else:
            B = _log_int(rng, 1, 16)
            c.update(B=B, S=_log_int(rng, 1, max(1, min(16384, room // B))))
        return c
    c.update(page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, rng.randint(1, 40)]), zero=rng.choice([0, 0, 1]), Hkv=rng.choice([1, 2, 4, 8, 16, 32]))
    if op == "append":
        B = _log_int(rng, 1, 256)
        G = rng.choice([0, 1, 2, 4, 8])
        room = 16384 * 8 * 128 * 6 // (c["Hkv"] * D * (2 + max(1, G)))
        hi = _log_int(rng, 1, max(1, min(16384, room // B)))
        c.update(B=B, G=G, lo=0, hi=_log_int(rng, 1, 2000), nlo=1, nhi=hi, **turn)
        return c
    G = rng.choice([1, 2, 3, 4, 8, 16])
    B = _log_int(rng, 1, 48)
    nhi = _log_int(rng, 1, 4096)
    keys = int(ONE_CALL / (4.0 * B * nhi * G * c["Hkv"] * D))  # a sequence's, for the largest listed work
    if keys < 64:
        nhi = max(1, nhi * keys // 64)
        keys = 64
    hi = _log_int(rng, 1, max(1, min(65536, keys, 300_000_000 // (B * c["Hkv"] * D))))
    c.update(B=B, G=G, lo=rng.choice([0, 1, hi]), hi=hi, nlo=rng.choice([1, nhi]), nhi=nhi)
    return c


def _lens(case):
    """The sequences' cached and new lengths: log-uniform, the last `zero` of them empty."""
    rng = random.Random(case["mix"])
    pick = lambda lo, hi: hi if lo >= hi else max(lo, min(hi, _log_int(rng, lo + 1, hi + 1) - 1))  # noqa: E731
    cached = [pick(case["lo"], case["hi"]) for _ in range(case["B"])]
    new = [pick(case["nlo"], case["nhi"]) for _ in range(case["B"])]
    for i in range(min(case["zero"], case["B"] - 1)):
        cached[-1 - i] = new[-1 - i] = 0
    return cached, new


def _pages(n, page):
    return -(-n // page)


def work(case):
    D = case["D"]
    if case["op"] == "rope":
        T = case["T"] if case["form"] == "packed" else case["B"] * case["S"]
        n = T * (case["Hq"] + case["Hk"])
        return {"bytes": n * D * 4 + (4 * T if case["form"] == "packed" else 0) + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    cached, new = _lens(case)
    page, Hkv, G = case["page"], case["Hkv"], case["G"]
    if case["op"] == "append":
        T = max(1, sum(new) + case["pad"])
        runs = sum(_pages(c + n, page) - c // page for c, n in zip(cached, new) if n)
        bytes_ = sum(new) * Hkv * D * (4 + 2) + T * 8 + runs * Hkv * 8 + T * Hkv * G * D * 4 + 4 * case["rot"]
        return {"bytes": bytes_, "flops": 8 * sum(new) * Hkv * D + 3 * (sum(new) * Hkv + T * Hkv * G) * case["rot"]}
    seen = sum(n * c + n * (n + 1) // 2 for c, n in zip(cached, new))
    keys = sum(c + n for c, n in zip(cached, new) if n)
    pages = sum(_pages(c + n, page) for c, n in zip(cached, new) if n)
    rows = sum(new) * Hkv * G
    return {"bytes": keys * Hkv * D * 2 + pages * (8 * Hkv + 4) + rows * (4 * D + 4), "flops": 4 * seen * Hkv * G * D}


# ----------------------------------------------------------------- inputs
BASE = 10000.0
SPAN = 4096  # positions that the unstretched frequencies were made for


def _frequencies(case):
    """Radians a position of each pair, and the amplitude: base^(-2i/rot), and with `yarn` = s the pairs that make fewer than one turn over
    SPAN positions s times slower, those with more than 32 as they are, in between a mixture; amplitude 0.1 ln s + 1."""
    rot, s = case["rot"], case["yarn"]
    f = [BASE ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not s:
        return f, 1.0
    at = lambda turns: rot * math.log(SPAN / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731  (the pair that makes so many turns)
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
    return [x * (1 - r) + x / s * r for x, r in zip(f, ramp)], 0.1 * math.log(s) + 1.0


def _phases(case, dev):
    """The frequencies in units of 2^-64 of a turn (whole numbers modulo 2^64, as int64)."""
    f, amplitude = _frequencies(case)
    steps = [int(x / (2 * math.pi) * 2.0 ** 64) % (1 << 64) for x in f]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in steps], dtype=torch.int64, device=dev), amplitude


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s, 1 for amax = 0."""
    m, e = torch.frexp(amax)  # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 2^9
    e = e - 9 + (m > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-100, 120)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _table(case, g, dev):
    """The block table with the step's pages, and how many pages the cache has."""
    cached, new = _lens(case)
    have = [_pages(c + n, case["page"]) for c, n in zip(cached, new)]
    width, num_pages = max(1, max(have)) + 2, sum(have) + 8
    ids = torch.randperm(num_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((case["B"], width), -1, dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev)[None, :] < torch.tensor(have, device=dev)[:, None]] = ids[: sum(have)]
    return table, num_pages


def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    D = case["D"]
    s = dict(op=case["op"], D=D)
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)  # noqa: E731
    if case["op"] == "rope":
        Hq, Hk = case["Hq"], case["Hk"]
        phases, amplitude = _phases(case, dev)
        s.update(phases=phases, amplitude=amplitude, inter=case["inter"], inverse=case["form"] == "grad", positions=None)
        if case["form"] == "packed":
            T = case["T"]
            fused = normal(T, (Hq + 2 * Hk) * D)
            s.update(q=fused[:, : Hq * D].unflatten(1, (Hq, D)), k=fused[:, Hq * D: (Hq + Hk) * D].unflatten(1, (Hk, D)),
                     positions=torch.randint(case["lo"], case["hi"] + 1, (T,), generator=g, device=dev, dtype=torch.int32),
                     q_out=torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=dev), k_out=torch.zeros((T, Hk, D), dtype=torch.bfloat16, device=dev))
            return s
        B, S = case["B"], case["S"]
        heads = lambda t, a, n: t[:, :, a * D: (a + n) * D].unflatten(2, (n, D)).transpose(1, 2)  # noqa: E731  [B, n, S, D], a view
        if case["form"] == "train":
            fused = normal(B, S, (Hq + 2 * Hk) * D)
            s.update(q=heads(fused, 0, Hq), k=heads(fused, Hq, Hk), q_out=torch.zeros((B, Hq, S, D), dtype=torch.bfloat16, device=dev),
                     k_out=torch.zeros((B, Hk, S, D), dtype=torch.bfloat16, device=dev))
        else:
            fused = torch.zeros((B, S, (Hq + 2 * Hk) * D), dtype=torch.bfloat16, device=dev)
            s.update(q=normal(B, Hq, S, D), k=normal(B, Hk, S, D), q_out=heads(fused, 0, Hq), k_out=heads(fused, Hq, Hk))
        return s

    cached, new = _lens(case)
    page, B, Hkv, G = case["page"], case["B"], case["Hkv"], case["G"]
    T = max(1, sum(new) + case["pad"])
    table, num_pages = _table(case, g, dev)
    if case["op"] == "append":
        phases, amplitude = _phases(case, dev)
        n, c = torch.tensor(new, device=dev), torch.tensor(cached, device=dev)
        seq = torch.repeat_interleave(torch.arange(B, device=dev), n)
        pos = c[seq] + torch.arange(seq.numel(), device=dev) - (torch.cumsum(n, 0) - n)[seq]
        slots = torch.full((T,), -1, dtype=torch.int32, device=dev)
        positions = torch.zeros((T,), dtype=torch.int32, device=dev)
        slots[: seq.numel()] = table[seq, pos // page] * page + (pos % page).to(torch.int32)
        positions[: seq.numel()] = pos.to(torch.int32)
        wide = (G + 2) * Hkv * D
        fused = torch.randn((T, wide), generator=g, device=dev)
        fused *= torch.exp(0.5 * torch.randn((wide,), generator=g, device=dev))  # channels differ in size
        fused = fused.to(torch.bfloat16)
        codes = lambda: normal(num_pages, Hkv, page, D).mul_(100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)  # noqa: E731
        scales = lambda: torch.randint(127 - 9, 127 - 6, (num_pages, Hkv), generator=g, device=dev, dtype=torch.int32).mul_(1 << 23).view(torch.float32)  # noqa: E731
        at = G * Hkv * D
        s.update(page=page, phases=phases, amplitude=amplitude, inter=case["inter"], slots=slots, positions=positions,
                 k=fused[:, at: at + Hkv * D].unflatten(1, (Hkv, D)), v=fused[:, at + Hkv * D:].unflatten(1, (Hkv, D)),
                 k_pages=codes(), v_pages=codes(), k_scale=scales(), v_scale=scales(), q=None, q_out=None,
                 runs=max(1, sum(_pages(a + b, page) - a // page for a, b in zip(cached, new) if b)))
        if G:
            s.update(q=fused[:, :at].unflatten(1, (G * Hkv, D)), q_out=torch.zeros((T, G * Hkv, D), dtype=torch.bfloat16, device=dev))
        return s

    Hq = Hkv * G
    fused = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=dev).mul_(1.5).to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)

    def pages():
        codes = torch.empty((num_pages, Hkv, page, D), dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty((num_pages, Hkv), device=dev)
        size = torch.exp(0.4 * torch.randn((Hkv, 1, D), generator=g, device=dev))  # channels differ in size
        step = max(1, (1 << 26) // (Hkv * page * D))
        for i in range(0, num_pages, step):
            x = torch.randn((min(step, num_pages - i), Hkv, page, D), generator=g, device=dev) * size
            sc = _pow2_scale(x.abs().amax((2, 3)))
            codes[i: i + step] = (x / sc[:, :, None, None]).to(torch.float8_e4m3fn)
            scale[i: i + step] = sc
        return codes, scale

    kp, ks = pages()
    vp, vs = pages()
    s.update(page=page, cached=cached, new=new, q=fused[:, : Hq * D].unflatten(1, (Hq, D)), cu=_i32(cu, dev), lens=_i32([c + n for c, n in zip(cached, new)], dev),
             table=table, k_pages=kp, v_pages=vp, k_scale=ks, v_scale=vs, scale=D ** -0.5, o=torch.zeros((T, Hq, D), dtype=torch.bfloat16, device=dev),
             lse=torch.zeros((T, Hq), device=dev), workspace=torch.empty(SCRATCH, dtype=torch.uint8, device=dev))
    return s


# ------------------------------------------------------------ plain forms
def _turned(x, positions, phases, amplitude, interleaved, inverse=False):
    """x [..., tokens, D] in 32 bits, its first 2 * len(phases) elements rotated; positions [tokens] or [..., tokens]."""
    angle = (positions.long()[..., None] * phases).double() * (math.pi / 2.0 ** 63)  # the product wraps around: whole turns drop out
    cos, sin = (torch.cos(angle) * amplitude).float(), (torch.sin(angle) * amplitude).float()
    if inverse:
        sin = -sin
    half = phases.numel()
    x = x.float()
    if interleaved:
        a, b = x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half: 2 * half]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _rope(s):
    packed = s["q"].dim() == 3
    for name in ("q", "k"):
        x = s[name].transpose(0, 1) if packed else s[name]
        positions = s["positions"] if s["positions"] is not None else torch.arange(x.shape[-2], device=x.device)
        y = _turned(x, positions, s["phases"], s["amplitude"], s["inter"], s["inverse"])
        s[name + "_out"].copy_(y.transpose(0, 1) if packed else y)
    return dict(q=s["q_out"], k=s["k_out"])


def _append(s):
    page, R, slots = s["page"], s["runs"], s["slots"].long()
    T, dev = slots.numel(), slots.device
    there = slots >= 0
    first = there & (torch.cat([slots.new_full((1,), -1), slots[:-1]]) // page != slots // page)
    run = torch.where(there, torch.cumsum(first.long(), 0) - 1, R)  # tokens without a place go behind the last run
    of_run = torch.zeros(R + 1, dtype=torch.long, device=dev).scatter_(0, run, slots.clamp(min=0) // page)[:R]
    start = torch.full((R + 1,), page, dtype=torch.long, device=dev).scatter_reduce_(0, run, slots % page, "amin")[:R]
    count = torch.zeros(R + 1, dtype=torch.long, device=dev).scatter_add_(0, run, torch.ones_like(run))[:R]
    row = torch.arange(page, device=dev)
    old = (row < start[:, None])[:, None, :, None]
    begin = torch.full((R + 1,), T, dtype=torch.long, device=dev).scatter_reduce_(0, run, torch.arange(T, device=dev), "amin")[:R]
    token = (begin[:, None] + row - start[:, None]).clamp(0, T - 1)
    fresh = ((row >= start[:, None]) & (row < (start + count)[:, None]))[:, None, :, None]

    def write(x, pages, scales):
        x = x[:, token].transpose(0, 1)  # [R, Hkv, page, D]
        amax = torch.where(fresh & torch.isfinite(x), x.abs(), 0.0).amax((2, 3))
        was = scales[of_run]
        scale = torch.where(start[:, None] > 0, torch.maximum(was, _pow2_scale(amax)), _pow2_scale(amax))
        codes = pages[of_run]
        kept = codes.float() * (was / scale)[:, :, None, None]
        put = torch.where(x.isnan(), x, (x / scale[:, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX))
        codes = torch.where(fresh, put.to(torch.float8_e4m3fn).float(), torch.where(old, kept.to(torch.float8_e4m3fn).float(), codes.float()))
        pages.view(torch.uint8)[of_run] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[of_run] = scale

    turn = lambda x: _turned(x.transpose(0, 1), s["positions"], s["phases"], s["amplitude"], s["inter"])  # noqa: E731  [heads, T, D]
    write(turn(s["k"]), s["k_pages"], s["k_scale"])
    write(s["v"].transpose(0, 1).float(), s["v_pages"], s["v_scale"])
    if s["q"] is not None:
        s["q_out"].copy_(turn(s["q"]).transpose(0, 1))
    return {n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale", "q_out") if s[n] is not None}


def _chunk(s):
    page, dev = s["page"], s["q"].device
    Hkv, D = s["k_pages"].shape[1], s["D"]
    G = s["q"].shape[1] // Hkv
    t = 0
    for b, (c, n) in enumerate(zip(s["cached"], s["new"])):
        if not n:
            continue
        at = s["table"][b, : _pages(c + n, page)].long()
        hidden = torch.arange(c + n, device=dev) > (c + torch.arange(n, device=dev))[:, None]
        for h in range(Hkv):
            k, v = ((codes.view(torch.uint8)[at, h].view(torch.float8_e4m3fn).float() * scale[at, h][:, None, None]).flatten(0, 1)[: c + n]
                    for codes, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            x = s["q"][t: t + n, h * G: h * G + G].float().transpose(0, 1)  # [G, n, D]
            sc = (x @ k.T).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
            m = sc.amax(2, keepdim=True)
            p = sc.sub_(m).exp_()
            total = p.sum(2, keepdim=True)
            s["o"][t: t + n, h * G: h * G + G] = ((p @ v) / total).transpose(0, 1).to(torch.bfloat16)
            s["lse"][t: t + n, h * G: h * G + G] = (torch.log(total) + m)[..., 0].T
        t += n
    return dict(o=s["o"], lse=s["lse"])


def run(s):
    if own:
        import exact_attention_82_gb300 as fa

        if s["op"] == "rope":
            turn = fa.fa_rope_bwd if s["inverse"] else fa.fa_rope
            q, k = turn(s["q"], s["k"], s["phases"], positions=s["positions"], interleaved=s["inter"], amplitude=s["amplitude"], q_out=s["q_out"], k_out=s["k_out"])
            return dict(q=q, k=k)
        if s["op"] == "append":
            fa.fa_kv_append_rope(s["k"], s["v"], s["positions"], s["phases"], s["slots"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], q=s["q"],
                                 q_out=s["q_out"], interleaved=s["inter"], amplitude=s["amplitude"])
            return {n: s[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale", "q_out") if s[n] is not None}
        o, lse = fa.fa_fwd_paged_chunk(s["q"], s["cu"], s["lens"], s["table"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], o=s["o"], lse=s["lse"],
                                       scale=s["scale"], workspace=s["workspace"])
        return dict(o=o, lse=lse)
    return {"rope": _rope, "append": _append, "chunk": _chunk}[s["op"]](s)


# ------------------------------------------- the definition, in 64 bits
def _two_to(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(y):
    """y rounded to the nearest e4m3 value, ties to even, held to +-448."""
    y = y.clamp(-E4M3_MAX, E4M3_MAX)
    e = (torch.frexp(y).exponent - 1).clamp(min=-6)
    step = _two_to(torch.where(y == 0, -6, e) - 3)
    return torch.round(y / step) * step


def _exact_turned(case, x, positions, sign=1.0):
    """x [..., D] rotated, as a product of complex numbers, from the frequencies themselves; positions broadcast against x[..., 0]."""
    f, amplitude = _frequencies(case)
    rot = case["rot"]
    angle = positions.double()[..., None] * torch.tensor(f, dtype=torch.float64, device=x.device)
    factor = torch.polar(torch.full_like(angle, amplitude), sign * angle)
    y = x.double().clone()
    re, im = (slice(0, rot, 2), slice(1, rot, 2)) if case["inter"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(y[..., re], y[..., im]) * factor
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        out = {}
        for name in ("q", "k"):
            x = s[name]
            at = s["positions"][:, None] if s["positions"] is not None else torch.arange(x.shape[-2], device=x.device)
            out[name] = _exact_turned(case, x, at, -1.0 if s["inverse"] else 1.0)
        return out
    cached, new = _lens(case)
    page = case["page"]
    if case["op"] == "append":
        out = {}
        slots = s["slots"].tolist()
        turned = _exact_turned(case, s["k"], s["positions"][:, None])
        for name, x in (("k", turned), ("v", s["v"].double())):
            codes, scales, t = s[name + "_pages"].double(), s[name + "_scale"].double(), 0
            for c, n in zip(cached, new):
                while n:
                    p, r = divmod(slots[t], page)
                    m = min(n, page - r)
                    y = x[t: t + m].transpose(0, 1)
                    amax = y.abs().amax((1, 2))
                    scale = _two_to(torch.frexp(amax / 512.0).exponent)  # amax < 512 scale
                    scale = torch.where(scale * (E4M3_MAX / 2) >= amax, scale / 2, torch.where(scale * E4M3_MAX < amax, 2 * scale, scale))
                    if r:
                        scale = torch.maximum(scale, scales[p])
                        codes[p, :, :r] = _round_e4m3(codes[p, :, :r] * (scales[p] / scale)[:, None, None])
                    codes[p, :, r: r + m] = _round_e4m3(y / scale[:, None, None])
                    scales[p] = scale
                    t, n = t + m, n - m
            out[name + "_pages"], out[name + "_scale"] = codes, scales
        out = {n: out[n] for n in ("k_pages", "v_pages", "k_scale", "v_scale")}
        if s["q"] is not None:
            out["q_out"] = _exact_turned(case, s["q"], s["positions"][:, None])
        return out
    if work(case)["flops"] > 4e12:
        return None
    G = case["G"]
    o, lse = s["o"].double(), s["lse"].double()
    t, dev = 0, o.device
    for b, (c, n) in enumerate(zip(cached, new)):
        for h in range(case["Hkv"] if n else 0):
            at = s["table"][b, : _pages(c + n, page)].long()
            j = torch.arange(at.numel() * page, device=dev)
            k = (s["k_pages"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double() * s["k_scale"][at, h].double()[:, None, None]).flatten(0, 1)
            v = (s["v_pages"].view(torch.uint8)[at, h].view(torch.float8_e4m3fn).double() * s["v_scale"][at, h].double()[:, None, None]).flatten(0, 1)
            for i in range(0, n, 256):  # a few tokens at a time: 64-bit scores are large
                m = min(256, n - i)
                x = s["q"][t + i: t + i + m, h * G: (h + 1) * G].double()
                sc = (x @ k.T) * s["scale"]
                sc.masked_fill_(j > (c + i + torch.arange(m, device=dev))[:, None, None], -math.inf)
                o[t + i: t + i + m, h * G: (h + 1) * G] = torch.softmax(sc, 2) @ v
                lse[t + i: t + i + m, h * G: (h + 1) * G] = torch.logsumexp(sc, 2)
        t += n
    return dict(o=o, lse=lse)
