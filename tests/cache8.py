"""Plain 64-bit model of the e4m3 paged cache, shared by its GPU tests: quantisation of blocks,
appending, attention, and a builder of caches with poisoned unused places."""
import math

import numpy as np
import torch


def e4m3_values() -> np.ndarray:
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


VALUES = e4m3_values()


def round_e4m3(x):
    """Code of the nearest e4m3 value of finite x (|x| <= 448), ties to the even code."""
    a = np.abs(x)
    pos = VALUES[:127]  # 0 .. 448
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


def need_scale(amax):
    """Least power of two s >= 2^-126 with amax <= 448 s; 0 for 0; NaN for what is not finite."""
    if not math.isfinite(amax):
        return math.nan
    if amax == 0:
        return 0.0
    m, e = math.frexp(amax)
    return math.ldexp(1.0, max(e - 9 if m <= 0.875 else e - 8, -126))


def append(codes, scales, x, table, lens, cu, sb):
    """In place on host copies: codes [P, ps, H, d] uint8, scales [P, H, nb] float64, x float64."""
    ps, H = codes.shape[1], codes.shape[2]
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        old = lens[b] - n
        for blk in range(old // sb, (lens[b] + sb - 1) // sb if n else 0):
            page, r0 = table[b, blk * sb // ps], blk * sb % ps
            lo, hi = max(old, blk * sb), min(lens[b], (blk + 1) * sb)
            rows = x[cu[b] + lo - old:cu[b] + hi - old]
            for h in range(H):
                top = np.abs(rows[:, h])
                need = need_scale(float(np.max(top)) if np.all(np.isfinite(top)) else math.nan)
                had = float(scales[page, h, r0 // sb]) if blk * sb < old else 0.0
                s = math.nan if math.isnan(need) or math.isnan(had) else max(need, had)
                held = slice(r0, r0 + max(0, lo - blk * sb))
                if s > had:
                    codes[page, held, h] = round_e4m3(VALUES[codes[page, held, h]] * (had / s))
                put = slice(r0 + lo - blk * sb, r0 + hi - blk * sb)
                if math.isnan(s):
                    codes[page, put, h] = 0x7F
                elif s == 0:
                    codes[page, put, h] = 0
                else:
                    codes[page, put, h] = round_e4m3(rows[:, h] / s)
                scales[page, h, r0 // sb] = s


def gather(codes, scales, table_row, n, sb):
    """The first n rows of a sequence as values, [n, H, d]."""
    ps, H, d = codes.shape[1:]
    j = np.arange(n)
    page, r = table_row[j // ps].astype(np.int64), j % ps
    return VALUES[codes[page, r]] * scales[page, :, r // sb][:, :, None]


def attend(q, kc, ks, vc, vs, table, lens, sb, scale):
    """o, lse and the bounds' ingredients for q [B, Nq, Hq, d] in 64 bits."""
    B, Nq, Hq, d = q.shape
    H = kc.shape[2]
    G = Hq // H
    o, lse = np.zeros(q.shape), np.full((B, Hq, Nq), -np.inf)
    o_abs, v_sum, t_abs = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, Hq, Nq))
    for b in range(B):
        if lens[b] == 0:
            continue
        k, v = gather(kc, ks, table[b], lens[b], sb), gather(vc, vs, table[b], lens[b], sb)
        for i in range(Nq):
            n = lens[b] - Nq + 1 + i
            if n <= 0:
                continue
            for h in range(Hq):
                t = k[:n, h // G] @ q[b, i, h] * scale
                m = t.max()
                p = np.exp(t - m)
                z = p.sum()
                vv = v[:n, h // G]
                o[b, i, h] = p @ vv / z
                o_abs[b, i, h] = p @ np.abs(vv) / z
                v_sum[b, i, h] = np.abs(vv).sum(0) / max(z, 1.0)
                t_abs[b, h, i] = (np.abs(k[:n, h // G]) @ np.abs(q[b, i, h])).max() * scale
                lse[b, h, i] = m + math.log(z)
    return o, lse, o_abs, v_sum, t_abs


def build(rng, lens, ps, sb, H, d, extra=2, spread=2.0):
    """A filled cache: (kc, ks, vc, vs, table), codes uint8, scales float64, the unused rows and
    pages holding NaN codes and NaN scales, unused table entries -1."""
    need = [(n + ps - 1) // ps for n in lens]
    P = sum(need) + extra
    order = rng.permutation(P)
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    out = [np.full((P, ps, H, d), 0x7F, np.uint8), np.full((P, H, ps // sb), np.nan),
           np.full((P, ps, H, d), 0x7F, np.uint8), np.full((P, H, ps // sb), np.nan)]
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    for w in (0, 2):
        x = rng.standard_normal((int(cu[-1]), H, d)) * np.exp2(rng.uniform(-spread, spread, (int(cu[-1]), H, 1)))
        append(out[w], out[w + 1], x.astype(np.float32).astype(np.float64), table, np.array(lens), cu, sb)
    return out[0], out[1], out[2], out[3], table


def to_device(kc, ks, vc, vs, table, lens):
    dev = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return (dev(kc).view(torch.float8_e4m3fn), dev(ks.astype(np.float32)), dev(vc).view(torch.float8_e4m3fn),
            dev(vs.astype(np.float32)), dev(table.astype(np.int32)), dev(np.array(lens, np.int32)))
