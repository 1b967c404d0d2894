"""Plain 64-bit forms of the operators over the 8-bit cache and of block eviction, and the error
bounds that their kernels are held to.  CPU tensors, loops, no code of the package."""
import math

import numpy as np
import torch

BLOCK, D, N_SEL, N_LOCAL = 32, 128, 16, 4
E4M3 = torch.float8_e4m3fn


def grid():
    """The 256 values of e4m3 (1 sign, 4 exponent bits of bias 7, 3 fraction bits, no infinity)."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return np.array(v)


GRID = grid()


def values(codes):
    """Codes (float8 tensor) as 64-bit values."""
    return torch.from_numpy(GRID[codes.cpu().view(torch.uint8).numpy()])


def encode(x):
    """64-bit values to e4m3 codes: nearest, ties to the even code, past 448 to 448, not finite to NaN."""
    x = np.asarray(x, dtype=np.float64)
    mag = GRID[:127]
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.minimum(np.searchsorted(mag, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = mag[hi] - a, a - mag[lo]
    c = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    c = np.where(np.signbit(x), c + 128, c)
    return np.where(np.isfinite(x), c, 127).astype(np.uint8)


def pow2_at_least(x):
    """The least power of two >= x, at least 2^-126."""
    m, e = math.frexp(x)
    return math.ldexp(1.0, max(-126, e - 1 if m == 0.5 else e)) if x > 0 else 2.0 ** -126


def need_scale(rows):
    a = np.abs(rows[np.isfinite(rows)])
    amax = float(a.max()) if a.size else 0.0
    s = 2.0 ** -126
    while amax > 448 * s:
        s *= 2
    return s


def make_pool(g, pages, H, scale_spread=0.5, odd_scale=False):
    """Random codes and scales.  odd_scale: scales that are not powers of two."""
    x = torch.randn((pages, H, BLOCK, D), generator=g) * torch.exp(scale_spread * torch.randn((pages, H, 1, 1), generator=g))
    amax = x.abs().amax(dim=(2, 3))
    s = amax / 448 if odd_scale else torch.exp2(torch.ceil(torch.log2(amax / 448)))
    return (x / s[:, :, None, None]).to(E4M3), s.float().contiguous()


def make_table(g, lens, max_blocks, spare=3):
    need = [-(-max(x, 0) // BLOCK) for x in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    t = torch.full((len(lens), max_blocks), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, pages


def attend(q, k, v, ks, vs, pages, blocks, p, scale):
    """One query row [H, 128] over the tokens t <= p of the given (page, block) lists, duplicates
    counted.  Returns out [H, 128], the weight of each listed block [H, n] and the bounds' inputs:
    the largest sum of |q k| (times the scales) and the largest |v| per head."""
    H = q.shape[0]
    n = len(blocks)
    if n == 0:
        return torch.zeros((H, D), dtype=torch.float64), torch.zeros((H, 0), dtype=torch.float64), torch.zeros(H), torch.zeros(H)
    pg = torch.tensor(pages, dtype=torch.long)
    kk = values(k[pg]) * ks[pg].double()[:, :, None, None]
    vv = values(v[pg]) * vs[pg].double()[:, :, None, None]
    tok = torch.tensor(blocks)[:, None] * BLOCK + torch.arange(BLOCK)[None]
    see = (tok <= p).reshape(-1)
    kk = kk.transpose(0, 1).reshape(H, n * BLOCK, D)[:, see]
    vv = vv.transpose(0, 1).reshape(H, n * BLOCK, D)[:, see]
    qd = q.double()
    z = torch.einsum("htd,hd->ht", kk, qd) * scale
    w = torch.softmax(z, dim=1)
    out = torch.einsum("ht,htd->hd", w, vv)
    full = torch.zeros((H, n * BLOCK), dtype=torch.float64)
    full[:, see] = w
    mag = (torch.einsum("htd,hd->ht", kk.abs(), qd.abs()) * abs(scale)).amax(dim=1)   # magnitudes: of the scale too
    return out, full.reshape(H, n, BLOCK).sum(-1), mag, vv.abs().amax(dim=(1, 2))


def weight_bound(mag):
    """Relative error of a softmax weight.  A score is 128 exact products summed in fp32 on the
    tensor cores in 8 steps of 16: at most 32 additions each off by 2^-23 of the sum of magnitudes
    (truncation counted, not half a step), so 2^-18 mag, then two fp32 products (2^-23 mag); exp2f
    is off by 2 units (2^-22), the fp32 sums of up to 2^12 weights in trees and chains of at most 64
    by 2^-18; the numerator and the denominator each carry that."""
    return 2 * (mag * (2.0 ** -18 + 2.0 ** -23) + 2.0 ** -22 + 2.0 ** -18)


def out_bound(out, mag, vmax, many=False):
    """bf16 output: half a step (2^-8 of the value) plus the weights' error times the largest value;
    the many-query form also rounds each weight and each partial output to fp16 (2^-11 each), with
    fp16's subnormals (2^-25) for up to 512 weights."""
    extra = 2.0 ** -10 + 512 * 2.0 ** -25 if many else 2.0 ** -20
    return out.abs() * 2.0 ** -8 + ((weight_bound(mag) + extra) * vmax)[:, None] * (1 + 2.0 ** -8) + 1e-38


def mass_bound(total, mag, queries=1):
    """Totals: each query's weight with its relative error (at most 1 in all), the fixed point of the
    many-query form (2^-41 each), one fp32 addition."""
    return queries * (weight_bound(mag) + 2.0 ** -40) + total.abs() * 2.0 ** -24


def evict(mass, table, lens, keep, sink):
    """Lists in place of tensors where that is plainer; returns the five outputs."""
    B, H, mb = mass.shape
    m, t, n = mass.clone(), table.clone(), lens.clone()
    freed = torch.full_like(table, -1)
    cut = torch.zeros_like(lens)
    for b in range(B):
        length = int(lens[b])
        nb = -(-length // BLOCK)
        if length < 0 or nb > mb or nb <= keep:
            continue
        total = mass[b].double().sum(0).tolist()
        cand = list(range(sink, nb - N_LOCAL))
        cand.sort(key=lambda j: (1, 0.0, j) if math.isnan(total[j]) else (0, -total[j], j))
        gone = sorted(cand[keep - sink - N_LOCAL:])
        out = set(gone)
        kept = [j for j in range(mb) if j not in out]
        m[b] = 0
        m[b, :, :len(kept)] = mass[b][:, kept]
        t[b] = -1
        t[b, :len(kept)] = table[b, kept]
        freed[b, :len(gone)] = table[b, gone]
        cut[b] = len(gone)
        n[b] = length - BLOCK * len(gone)
    return m, t, n, freed, cut


def rotate(x, tok, page):
    """page2d rotation of [..., 128] in 64 bits: 63 pairs by the token offset, one by the page's parity."""
    x = np.asarray(x, dtype=np.float64)
    ang = np.concatenate([np.array([float(tok) * 10000.0 ** (-i / 63) for i in range(63)]), [float(page % 2)]])
    c, s = np.cos(ang), np.sin(ang)
    a, b = x[..., :64], x[..., 64:]
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def append(state, starts, lens, table):
    """state: CPU tensors q, idx_q, k_new, v_new, idx_k_new, tok, page, k, v (codes), k_scale, v_scale,
    idx_k.  Returns the 64-bit q and idx_q (None rows where nothing is written) and the new caches."""
    n, H, _ = state["q"].shape
    q, idx_q = np.full((n, H, D), np.nan), np.full((n, D), np.nan)
    codes = {x: state[x].view(torch.uint8).numpy().copy() for x in "kv"}
    scale = {x: state[x + "_scale"].double().numpy().copy() for x in "kv"}
    idx_k = state["idx_k"].double().numpy().copy()
    wrote = np.zeros(idx_k.shape[:2], dtype=bool)
    pages = state["idx_k"].shape[0]
    for b, length in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        if a < 0 or e < a or e > n or length < e - a or length > table.shape[1] * BLOCK:
            continue
        p = length - (e - a)
        while p < length:
            end = min(length, p // BLOCK * BLOCK + BLOCK)
            toks = range(a + p - (length - (e - a)), a + end - (length - (e - a)))
            rot = []
            for i in toks:
                tk, pp = int(state["tok"][i]), int(state["page"][i])
                q[i] = rotate(state["q"][i].double(), tk, pp)
                idx_q[i] = rotate(state["idx_q"][i].double(), tk, pp)
                rot.append((rotate(state["k_new"][i].double(), tk, pp), state["v_new"][i].double().numpy(),
                            rotate(state["idx_k_new"][i].double(), tk, pp)))
            pg = int(table[b, p // BLOCK])
            if 0 <= pg < pages:
                r0 = p % BLOCK
                for which, name in ((0, "k"), (1, "v")):
                    rows = np.stack([r[which] for r in rot])           # [rows, H, D]
                    for h in range(H):
                        s = need_scale(rows[:, h])
                        if r0:
                            old = float(scale[name][pg, h])
                            s = max(s, pow2_at_least(old))
                            if s != old:
                                codes[name][pg, h, :r0] = encode(GRID[codes[name][pg, h, :r0]] * (old / s))
                        codes[name][pg, h, r0:r0 + len(toks)] = encode(rows[:, h] / s)
                        scale[name][pg, h] = s
                idx_k[pg, r0:r0 + len(toks)] = np.stack([r[2] for r in rot])
                wrote[pg, r0:r0 + len(toks)] = True
            p = end
    return {"q": q, "idx_q": idx_q, "k": codes["k"], "v": codes["v"], "k_scale": scale["k"], "v_scale": scale["v"],
            "idx_k": idx_k, "wrote": wrote}
