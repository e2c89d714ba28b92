"""The serving and long-context operators around the attention kernels: their measured cases,
their plain forms and their values in 64 bits.

Operators (`op` of a case):

* ``rope``    rotary positions of q and k in one call: half or interleaved pairs, the first
              ``rot`` columns of a head, frequencies scaled for long contexts; forward, and the
              backward that turns gradients back.
* ``append``  writes new K and V rows (bf16) into a paged cache held in 8 bits (e4m3) with one
              power-of-two scale per ``sb`` tokens and head, rescaling a block that grows.
* ``decode``  attention of 1..n new tokens per sequence over such a cache.
* ``fork``    copies, shares and frees the pages of a paged cache as sequences are forked or
              dropped: new block table, lengths, free pages, and the copied pages.
* ``compact`` moves the pages in use to the front of the pool and rewrites the block table.

Lengths and page placements follow from the case alone; all values follow from the seed.
"""
import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one step of 16 sequences in the middle of long contexts: launch latency
        dict(name="rope step", op="rope", B=16, N=1, Hq=64, Hkv=8, d=128, rot=128, layout="half", dtype="bf16",
             far=1000000, scaling="bands", factor=8.0, back=False),
        # the 8K prefill shape of the forward benchmark
        dict(name="rope prefill 8k", op="rope", B=1, N=8192, Hq=64, Hkv=8, d=128, rot=128, layout="half",
             dtype="bf16", far=0, scaling="none", factor=1.0, back=False),
        # training: gradients of a packed batch, part of the head, interleaved pairs
        dict(name="rope backward packed", op="rope", B=1, N=32749, Hq=32, Hkv=8, d=128, rot=64,
             layout="interleaved", dtype="bf16", far=0, scaling="linear", factor=4.0, back=True),
        # fp32 inputs of the tf32 forward, d = 64, an odd length
        dict(name="rope fp32 d64", op="rope", B=2, N=2047, Hq=12, Hkv=12, d=64, rot=32, layout="half",
             dtype="f32", far=5000, scaling="ntk", factor=2.0, back=False),
        # one new token for each of 16 sequences
        dict(name="append step", op="append", B=16, lo=1, hi=1, old=20000, Hkv=8, d=128, ps=16, sb=16, key=1),
        # the prompts of the packed forward benchmark go into the cache
        dict(name="append prompts", op="append", B=16, lo=256, hi=8192, old=100, Hkv=8, d=128, ps=64, sb=32, key=2),
        # a single short sequence: latency
        dict(name="decode short", op="decode", B=1, Nq=1, lo=37, hi=37, Hq=12, Hkv=12, d=64, ps=16, sb=16, key=3),
        # the ragged paged decode of the benchmark, in 8 bits
        dict(name="decode ragged", op="decode", B=16, Nq=1, lo=1, hi=32768, Hq=64, Hkv=8, d=128, ps=16, sb=16, key=4),
        # the 32K decode of the benchmark, larger pages
        dict(name="decode 32k", op="decode", B=8, Nq=1, lo=32768, hi=32768, Hq=64, Hkv=8, d=128, ps=64, sb=64, key=5),
        # verification of drafted tokens: five query tokens per sequence
        dict(name="decode drafted", op="decode", B=8, Nq=5, lo=500, hi=32768, Hq=64, Hkv=8, d=128, ps=32, sb=16, key=6),
        # parallel samples: 16 prompts become 64 sequences that share their full pages
        dict(name="fork samples", op="fork", B=16, R=64, lo=1, hi=16384, layers=4, Hkv=8, d=128, ps=64, sb=64,
             spare=1000, key=7),
        # half the pool was freed: the rest moves to the front
        dict(name="compact half", op="compact", B=32, lo=1, hi=16384, layers=2, Hkv=8, d=128, ps=64, sb=64,
             spare=4000, key=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "append", "decode", "decode", "decode", "fork", "compact"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 12])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    key = rng.randrange(10, 1 << 30)
    if op == "rope":
        B = rng.choice([1, 1, 2, 3, 16])
        room = 8192 * 72 * 128 // (B * Hkv * (G + 1) * d * 2)
        layout = rng.choice(["half", "interleaved"])
        return dict(op=op, B=B, N=_log_int(rng, 1, max(2, min(32768, room))), Hq=Hkv * G, Hkv=Hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4, 2 * rng.randrange(1, d // 2)]), layout=layout,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), far=rng.choice([0, 17, _log_int(rng, 1, 4000000)]),
                    scaling=rng.choice(["none", "linear", "ntk", "bands"]), factor=rng.choice([2.0, 4.0, 8.0, 32.0]),
                    back=rng.random() < 0.5)
    ps = rng.choice([16, 32, 64, 128, 256])
    sb = min(ps, rng.choice([16, 32, 64, 128, 256]))
    if op == "append":
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(2, 60000 // B))
        return dict(op=op, B=B, lo=max(1, hi // 16), hi=hi, old=rng.choice([0, 1, _log_int(rng, 1, 4000)]), Hkv=Hkv,
                    d=d, ps=ps, sb=sb, key=key)
    if op == "decode":
        B = _log_int(rng, 1, 32)
        Nq = rng.choice([1, 1, 1, 2, 3, 4, 8])
        hi = _log_int(rng, 8, max(9, min(32768, 8 * 32768 * 8 // (B * Hkv), 40000000 // (B * Hkv * G * Nq))))
        return dict(op=op, B=B, Nq=Nq, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, Hq=Hkv * G, Hkv=Hkv, d=d, ps=ps,
                    sb=sb, key=key)
    B = _log_int(rng, 1, 48)
    layers = rng.choice([1, 2, 3])
    c = dict(op=op, B=B, lo=1, hi=_log_int(rng, 2, max(3, min(32768, 7000000 // (B * Hkv * layers)))), layers=layers,
             Hkv=Hkv, d=d, ps=ps, sb=sb, spare=_log_int(rng, 80, 3000), key=key)
    if op == "fork":
        c["R"] = min(72, _log_int(rng, 1, 4 * B))
    return c


# ------------------------------------------------------------- what follows from the case
def _lengths(c):
    return np.random.RandomState(c["key"] % (1 << 31)).randint(c["lo"], c["hi"] + 1, c["B"]).astype(np.int64)


def _layout(c, lens, spare):
    """Block table (-1 in unused entries) over a shuffled pool, and the pool's size."""
    need = (lens + c["ps"] - 1) // c["ps"]
    total = int(need.sum()) + spare
    order = np.random.RandomState((c["key"] * 7 + 1) % (1 << 31)).permutation(max(total, 1))
    table = np.full((len(lens), max(1, int(need.max()))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += int(n)
    return table, max(total, 1)


def _parents(c):
    r = np.random.RandomState((c["key"] * 5 + 3) % (1 << 31))
    p = r.randint(0, c["B"], c["R"])
    p[r.rand(c["R"]) < 0.05] = -1  # a slot left empty
    return p.astype(np.int32)


def _old_new(c):
    """append: tokens held before, and new tokens, of each sequence."""
    r = np.random.RandomState((c["key"] * 3 + 2) % (1 << 31))
    return r.randint(0, c["old"] + 1, c["B"]).astype(np.int64), _lengths(c)


def _page_bytes(c):
    return c["ps"] * c["Hkv"] * c["d"] + c["Hkv"] * (c["ps"] // c["sb"]) * 4


def work(c):
    if c["op"] == "rope":
        es = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["N"]
        return dict(bytes=2 * n * (c["Hq"] + c["Hkv"]) * c["d"] * es + 4 * n,
                    flops=3 * n * (c["Hq"] + c["Hkv"]) * c["rot"])
    if c["op"] == "append":
        new = int(_old_new(c)[1].sum())
        return dict(bytes=2 * new * c["Hkv"] * c["d"] * 3 + 2 * new * c["Hkv"] * 4 / c["sb"],
                    flops=2 * new * c["Hkv"] * c["d"] * 3)
    if c["op"] == "decode":
        T = int(_lengths(c).sum())
        qo = c["B"] * c["Nq"] * c["Hq"] * (4 * c["d"] + 4)
        return dict(bytes=T * c["Hkv"] * (2 * c["d"] + 8 / c["sb"]) + 4 * T / c["ps"] + qo,
                    flops=4 * T * c["Nq"] * c["Hq"] * c["d"])
    lens = _lengths(c)
    need = (lens + c["ps"] - 1) // c["ps"]
    pair = 2 * c["layers"] * _page_bytes(c)  # K and V
    if c["op"] == "fork":
        p = _parents(c)
        seen, copies, rows = set(), 0, 0
        for x in p:
            if x >= 0:
                copies += int(x in seen and lens[x] % c["ps"] != 0)
                rows += int(need[x])
                seen.add(x)
        pages = int(need.sum()) + c["spare"]
        return dict(bytes=2 * copies * pair + 4 * (2 * rows + pages), flops=0)
    table, pages = _layout(c, lens, c["spare"])
    live = int(need.sum())
    return dict(bytes=2 * int((table >= live).sum()) * pair + 8 * live, flops=0)


# ------------------------------------------------------------------------------ inputs
def _rand(seed, n, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + n)
    return torch.randn(*shape, generator=g, device="cuda")


def _pow2_scale(amax):
    """The least power of two s with amax <= 448 s (0 for 0), not under 2^-126."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), torch.clamp(torch.where(m <= 0.875, e - 9, e - 8), min=-126))
    return torch.where(amax > 0, s, torch.zeros_like(s))


def _filled_pages(c, seed, n, pages):
    """A pool [pages, ps, Hkv, d] of e4m3 with its scales [pages, Hkv, ps / sb], whose heads and
    blocks differ in magnitude."""
    nb = c["ps"] // c["sb"]
    codes = torch.empty(pages, c["ps"], c["Hkv"], c["d"], dtype=E4M3, device="cuda")
    scales = torch.empty(pages, c["Hkv"], nb, device="cuda")
    step = max(1, (1 << 26) // (c["ps"] * c["Hkv"] * c["d"]))
    for at in range(0, pages, step):
        m = min(step, pages - at)
        x = _rand(seed, n + at * 16, m, nb, c["sb"], c["Hkv"], c["d"])
        x *= torch.exp2(_rand(seed, n + at * 16 + 1, m, nb, 1, c["Hkv"], 1) * 0.5)
        s = _pow2_scale(x.abs().amax(dim=(2, 4)))  # [m, nb, Hkv]
        codes[at:at + m] = (x / s[:, :, None, :, None]).to(E4M3).view(m, c["ps"], c["Hkv"], c["d"])
        scales[at:at + m] = s.transpose(1, 2)
    return codes, scales


def _frequencies(c):
    """Angular frequencies in 64 bits, [rot / 2]."""
    rot, theta, f = c["rot"], 10000.0, c["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "ntk" and rot > 2:
        theta = theta * f ** (rot / (rot - 2))
    w = theta ** (-2 * i / rot)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "bands":  # turns over 8192 positions: below 1 all scaled, above 32 none
        keep = ((8192 * w / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        w = w * (keep + (1 - keep) / f)
    return w


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "bands" else 1.0


def prepare(c, seed):
    s = dict(case=c)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    if c["op"] == "rope":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["q"] = _rand(seed, 1, c["B"], c["N"], c["Hq"], c["d"]).to(dt)
        s["k"] = _rand(seed, 2, c["B"], c["N"], c["Hkv"], c["d"]).to(dt)
        start = np.random.RandomState(seed % (1 << 31)).randint(0, c["far"] + 1, (c["B"], 1))
        s["positions"] = i32(start + np.arange(c["N"])[None])
        s["freqs"] = _frequencies(c)
        return s
    if c["op"] == "append":
        old, new = _old_new(c)
        table, pages = _layout(c, old + new, 3)
        s["k"] = _rand(seed, 1, int(new.sum()), c["Hkv"], c["d"]).bfloat16()
        s["v"] = (_rand(seed, 2, int(new.sum()), c["Hkv"], c["d"]) * 3).bfloat16()
        s["kp"], s["ks"] = _filled_pages(c, seed, 3, pages)
        s["vp"], s["vs"] = _filled_pages(c, seed, 5, pages)
        s["table"], s["lens"], s["new"] = i32(table), i32(old + new), i32(new)
        s["cu"] = i32(np.concatenate([[0], np.cumsum(new)]))
        return s
    lens = _lengths(c)
    if c["op"] == "decode":
        table, pages = _layout(c, lens, 3)
        s["q"] = _rand(seed, 1, c["B"], c["Nq"], c["Hq"], c["d"]).bfloat16()
        s["kp"], s["ks"] = _filled_pages(c, seed, 3, pages)
        s["vp"], s["vs"] = _filled_pages(c, seed, 5, pages)
        s["table"], s["lens"], s["longest"] = i32(table), i32(lens), int(lens.max())
        return s
    table, pages = _layout(c, lens, c["spare"])
    s["pools"] = []
    for layer in range(c["layers"]):
        for x in (0, 1):
            s["pools"] += _filled_pages(c, seed + 7919 * layer, 3 + 2 * x, pages)
    s["table"], s["lens"], s["pages"] = i32(table), i32(lens), pages
    if c["op"] == "fork":
        s["parent"] = i32(_parents(c))
    return s


# ---------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, rot, half, back):
    """Rotates the first `rot` columns; cos, sin [B, N, 1, rot / 2] in 32 bits."""
    f = x.float()
    if half:
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
    else:
        a, b = f[..., :rot:2], f[..., 1:rot:2]
    if back:
        sin = -sin
    y0, y1 = a * cos - b * sin, b * cos + a * sin
    y = torch.cat([y0, y1], -1) if half else torch.stack([y0, y1], -1).flatten(-2)
    return torch.cat([y, f[..., rot:]], -1).to(x.dtype)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[..., None, None] * s["freqs"]
    cos, sin = (angle.cos() * _amplitude(c)).float(), (angle.sin() * _amplitude(c)).float()
    return [_turn(x, cos, sin, c["rot"], c["layout"] == "half", c["back"]) for x in (s["q"], s["k"])]


def _places(s):
    """append: page, row in the page of each new token, and whether it starts a sequence's blocks."""
    n, ps = s["k"].shape[0], s["case"]["ps"]
    t = torch.arange(n, device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = t - s["cu"].long()[b] + (s["lens"] - s["new"]).long()[b]
    return s["table"].long()[b, pos // ps], pos % ps, (s["lens"] - s["new"]).long()[b] - pos


def _plain_append(s):
    c = s["case"]
    nb, sb = c["ps"] // c["sb"], c["sb"]
    page, row, back = _places(s)  # back: tokens to the sequence's old end (<= 0)
    block = page * nb + row // sb  # number of the block over the pool
    held = row % sb + back  # old tokens in the block
    for x, pages, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        P, H = pages.shape[0], c["Hkv"]
        amax = torch.zeros(P * nb, H, device="cuda")
        amax.index_reduce_(0, block, x.float().abs().amax(-1), "amax")
        touched = torch.zeros(P * nb, dtype=torch.bool, device="cuda")
        touched[block] = True
        keep = torch.zeros(P * nb, dtype=torch.long, device="cuda")
        keep[block] = held.clamp(min=0)
        was = scales.transpose(1, 2).reshape(P * nb, H)
        before = torch.where((keep > 0)[:, None], was, torch.zeros_like(was))
        now = torch.where(touched[:, None], torch.maximum(before, _pow2_scale(amax)), was)
        u = touched.nonzero()[:, 0]  # the old rows of the blocks that grew
        blocks = pages.view(torch.uint8).view(P * nb, sb, H, c["d"])
        codes = blocks[u].view(E4M3).float()
        ratio = torch.where(now[u] > 0, before[u] / now[u], torch.ones_like(now[u]))
        scaled = (codes * ratio[:, None, :, None]).to(E4M3).view(torch.uint8)
        old = torch.arange(sb, device="cuda")[None, :] < keep[u][:, None]
        blocks[u] = torch.where(old[:, :, None, None], scaled, blocks[u])
        to = now[block]
        y = torch.where(to[..., None] > 0, x.float() / to[..., None], torch.zeros_like(x, dtype=torch.float32))
        pages.view(torch.uint8)[page, row] = y.to(E4M3).view(torch.uint8)
        scales.copy_(now.view(P, nb, H).transpose(1, 2))
    return [s["kp"], s["ks"], s["vp"], s["vs"]]


def _gathered(s, pages, scales, dt):
    """[B, longest, Hkv, d]: the cache of each sequence, dequantised."""
    c = s["case"]
    t = s["table"].long().clamp(min=0)
    x = pages.view(torch.uint8)[t].view(E4M3).to(dt)  # [B, maxp, ps, Hkv, d]
    x = x * scales.to(dt)[t].transpose(2, 3).repeat_interleave(c["sb"], 2)[..., None]
    return x.flatten(1, 2)[:, :s["longest"]]


def _plain_decode(s):
    c = s["case"]
    B, N, G, L = c["B"], c["Nq"], c["Hq"] // c["Hkv"], s["longest"]
    k = _gathered(s, s["kp"], s["ks"], torch.float32).permute(0, 2, 3, 1)  # [B, Hkv, d, L]
    q = s["q"].float().view(B, N, c["Hkv"], G, c["d"]).permute(0, 2, 1, 3, 4).reshape(B, c["Hkv"], N * G, c["d"])
    x = (torch.matmul(q, k) * c["d"] ** -0.5).view(B, c["Hkv"], N, G, L)
    del k
    end = s["lens"].view(B, 1, 1, 1, 1) - N + torch.arange(1, N + 1, device="cuda").view(1, 1, N, 1, 1)
    seen = torch.arange(L, device="cuda") < end
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    v = _gathered(s, s["vp"], s["vs"], torch.float32)
    v = torch.where((torch.arange(L, device="cuda") < s["lens"][:, None])[..., None, None], v, torch.zeros_like(v))
    o = torch.matmul(p.view(B, c["Hkv"], N * G, L), v.transpose(1, 2)).view(B, c["Hkv"], N, G, c["d"])
    o = torch.where(z > 0, o / z, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(s["q"].shape)
    lse = (m + torch.log(z))[..., 0].permute(0, 1, 3, 2).reshape(B, c["Hq"], N)
    return [o.bfloat16(), lse]


def _plain_fork(s):
    ps, P = s["case"]["ps"], s["pages"]
    table, lens, parent = s["table"].long(), s["lens"].long(), s["parent"].long()
    R, M = parent.numel(), table.shape[1]
    n = torch.where(parent >= 0, lens[parent.clamp(min=0)], torch.zeros_like(parent))
    t = torch.arange(M, device="cuda")[None]
    rows = torch.where(t < ((n + ps - 1) // ps)[:, None], table[parent.clamp(min=0)], torch.full_like(t, -1))
    i = torch.arange(R, device="cuda")
    last, part = n // ps, n % ps != 0
    tail = torch.where(part, rows.gather(1, last.clamp(max=M - 1)[:, None])[:, 0], torch.full_like(n, P))
    # who keeps a page: -1 where it is full in some row, else the first row that ends in it
    mark = torch.full((P + 2,), R, device="cuda")
    mark.index_reduce_(0, tail, i, "amin")
    full = rows[t < last[:, None]]
    mark[full] = -1
    copy = part & (mark[tail] != i)
    free = (mark[:P] == R).nonzero()[:, 0]
    to = free[(copy.long().cumsum(0) - 1).clamp(min=0)]
    rows = torch.where((t == last[:, None]) & copy[:, None], to[:, None], rows)
    src, dst = tail[copy], to[copy]
    for x in s["pools"]:
        y = x.view(torch.uint8)
        y[dst] = y[src]
    count = copy.sum()
    left = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    k = torch.arange(P, device="cuda")
    rest = (k < free.numel() - count)
    left = torch.where(rest, free[(k + count).clamp(max=free.numel() - 1)].int(), left)
    return [rows.int(), n.int(), left, (free.numel() - count).int().view(1)] + s["pools"]


def _plain_compact(s):
    ps, P = s["case"]["ps"], s["pages"]
    table, lens = s["table"].long(), s["lens"].long()
    held = torch.arange(table.shape[1], device="cuda")[None] < ((lens + ps - 1) // ps)[:, None]
    live = torch.zeros(P, dtype=torch.bool, device="cuda")
    live[table[held]] = True
    count = live.sum()
    k = torch.arange(P, device="cuda")
    src = (live & (k >= count)).nonzero()[:, 0]
    dst = (~live & (k < count)).nonzero()[:, 0]
    to = k.clone()
    to[src] = dst
    for x in s["pools"]:
        y = x.view(torch.uint8)
        y[dst] = y[src]
    rows = torch.where(held, to[table.clamp(min=0)], torch.full_like(table, -1))
    return [rows.int(), count.int().view(1)] + s["pools"]


def run(s):
    c = s["case"]
    if own:
        from exact_io_aware_97_b200 import binding as fa
        if c["op"] == "rope":
            turn = fa.rope_backward if c["back"] else fa.rope
            return list(turn(s["q"], s["k"], s["freqs"], s["positions"], interleaved=c["layout"] == "interleaved",
                             amplitude=_amplitude(c)))
        if c["op"] == "append":
            fa.cache_append_fp8(s["k"], s["v"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"], s["cu"])
            return [s["kp"], s["ks"], s["vp"], s["vs"]]
        if c["op"] == "decode":
            return list(fa.decode_paged_fp8(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["table"], s["lens"]))
        if c["op"] == "fork":
            return list(fa.pages_fork(s["pools"], s["table"], s["lens"], s["parent"], c["ps"])) + s["pools"]
        return list(fa.pages_compact(s["pools"], s["table"], s["lens"], c["ps"])) + s["pools"]
    plain = dict(rope=_plain_rope, append=_plain_append, decode=_plain_decode, fork=_plain_fork, compact=_plain_compact)
    return plain[c["op"]](s)


# -------------------------------------------------------------------- values in 64 bits
def _exact_rope(s):
    """Each pair as a complex number times amplitude * exp(+-i angle)."""
    c = s["case"]
    h = c["rot"] // 2
    w = _frequencies(c)
    pos = s["positions"].to(torch.float64)
    turn = torch.polar(torch.full((c["B"], c["N"], h), _amplitude(c), dtype=torch.float64, device="cuda"),
                       pos[:, :, None] * w * (-1 if c["back"] else 1))
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        at = torch.arange(h, device="cuda")
        i0, i1 = (at, at + h) if c["layout"] == "half" else (2 * at, 2 * at + 1)
        z = torch.complex(y[..., i0], y[..., i1]) * turn[:, :, None]
        y[..., i0], y[..., i1] = z.real, z.imag
        out.append(y)
    return out


def _nearest_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even, in 64 bits (|x| <= 448)."""
    e = torch.frexp(x)[1].double() - 1
    step = torch.exp2(torch.clamp(e, min=-6.0) - 3)
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    sb, out = c["sb"], []
    table, lens, new, cu = (s[n].cpu().numpy() for n in ("table", "lens", "new", "cu"))
    for x, pages, scales in ((s["k"], s["kp"], s["ks"]), (s["v"], s["vp"], s["vs"])):
        codes, sc = pages.float().double(), scales.double()
        flat = codes.view(-1, c["Hkv"], c["d"])  # rows of the pool
        for b in range(c["B"]):
            lo, hi = int(lens[b] - new[b]), int(lens[b])
            if hi == lo:
                continue
            first = lo // sb * sb
            n = -(-(hi - first) // sb) * sb
            pos = np.arange(first, first + n)
            rows = table[b][np.minimum(pos // c["ps"], table.shape[1] - 1)].astype(np.int64) * c["ps"] + pos % c["ps"]
            rows = torch.from_numpy(rows).cuda()
            pos = torch.from_numpy(pos).cuda()
            page, blk = rows[::sb] // c["ps"], rows[::sb] % c["ps"] // sb
            val = torch.zeros(n, c["Hkv"], c["d"], dtype=torch.float64, device="cuda")
            isnew = (pos >= lo) & (pos < hi)
            val[isnew] = x[int(cu[b]):int(cu[b + 1])].double()
            top = val.view(-1, sb, c["Hkv"], c["d"]).abs().amax(dim=(1, 3))
            need = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-40) / 448))), 0.0)
            had = sc[page, :, blk] * (pos[::sb] < lo)[:, None]
            got = torch.maximum(need, had)
            sc[page, :, blk] = got
            per, was = (y.repeat_interleave(sb, 0)[..., None] for y in (got, had))
            val = torch.where((pos < lo)[:, None, None], flat[rows] * was, val)
            val = torch.where(per > 0, _nearest_e4m3(val / per.clamp(min=1e-300)), 0.0)
            put = pos < hi
            flat[rows[put]] = val[put]
        out += [codes, sc]
    return out


def _exact_decode(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hq"], c["Nq"]), -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for b in range(c["B"]):
        pg = s["table"][b, :-(-lens[b] // c["ps"])].long()
        kv = []
        for pages, scales in ((s["kp"], s["ks"]), (s["vp"], s["vs"])):
            y = pages.view(torch.uint8)[pg].view(E4M3).double()
            f = torch.repeat_interleave(scales[pg].double(), c["sb"], dim=2).permute(0, 2, 1)
            kv.append((y * f[..., None]).reshape(-1, c["Hkv"], c["d"]))
        for i in range(c["Nq"]):
            n = lens[b] - c["Nq"] + 1 + i
            if n <= 0:
                continue
            q = s["q"][b, i].double().view(c["Hkv"], G, c["d"])
            x = torch.einsum("hgd,jhd->hgj", q, kv[0][:n]) / math.sqrt(c["d"])
            lse[b, :, i] = torch.logsumexp(x, -1).flatten()
            o[b, i] = torch.einsum("hgj,jhd->hgd", torch.softmax(x, -1), kv[1][:n]).reshape(c["Hq"], c["d"])
    return [o, lse]


def exact(c, seed):
    # fork and compact only move values: nothing of theirs is computed
    if c["op"] not in ("rope", "append", "decode"):
        return None
    return dict(rope=_exact_rope, append=_exact_append, decode=_exact_decode)[c["op"]](prepare(c, seed))
