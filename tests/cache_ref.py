"""The 8-bit cache's operators in 64 bits (numpy), one sequence and one head at a time, for the tests."""
import math

import numpy as np
import torch

BLOCK = 32
QMAX = {"e4m3": 448.0, "int8": 127.0}
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def e4m3_values():
    """The 256 numbers of the 1-4-3 format (NaN at 0x7f and 0xff), from its definition."""
    out = np.zeros(256)
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        v = float("nan") if (e, f) == (15, 7) else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        out[c] = -v if s else v
    return out


_E4M3 = e4m3_values()
_E4M3_POS = _E4M3[:127]              # 0 .. 448, ascending


def scale_of(amax, fmt):
    e = -126
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def to_code_value(x, fmt):
    """fp64 numbers to the nearest code's number, ties to even (within the range)."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.rint(x)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_E4M3_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _E4M3_POS[lo], _E4M3_POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.copysign(_E4M3_POS[pick], x)


def code_values(t):
    """A code tensor's numbers (without the scale) in fp64."""
    return t.detach().cpu().float().double().numpy()


def append(codes, scale, lengths, counts, x, fmt):
    """codes [B, cap, H, d] (numbers), scale [B, blocks, H], x [B, n, H, d]: the cache after the append."""
    codes, scale = codes.copy(), scale.copy()
    B, cap, H, d = codes.shape
    for b in range(B):
        start = lengths[b] - counts[b]
        for j in range(cap // BLOCK):
            rows = [s for s in range(j * BLOCK, (j + 1) * BLOCK) if start <= s < lengths[b]]
            if not rows:
                continue
            old = [s for s in range(j * BLOCK, (j + 1) * BLOCK) if s < start]
            for h in range(H):
                new = np.stack([x[b, s - start, h] for s in rows]).astype(np.float64)
                fin = np.abs(new[np.isfinite(new)])
                sc = scale_of(fin.max() if fin.size else 0.0, fmt)
                if old:
                    before = scale[b, j, h]
                    if before >= sc:
                        sc = before
                    else:
                        codes[b, old, h] = to_code_value(codes[b, old, h] * (before / sc), fmt)
                y = new / sc
                v = to_code_value(np.clip(np.nan_to_num(y, nan=0.0, posinf=QMAX[fmt], neginf=-QMAX[fmt]),
                                          -QMAX[fmt], QMAX[fmt]), fmt)
                if fmt == "e4m3":
                    v = np.where(np.isnan(new), np.nan, v)
                codes[b, rows, h] = v
                scale[b, j, h] = sc
    return codes, scale


def quantize(x, fmt):
    """Codes and scales of x [B, T, H, d] (T a multiple of 32) as torch tensors."""
    B, T, H, d = x.shape
    n = [T] * B
    codes, scale = append(np.zeros((B, T, H, d)), np.zeros((B, T // BLOCK, H)), n, n, x.double().numpy(), fmt)
    return torch.tensor(codes).to(torch.float32).to(DTYPE[fmt]), torch.tensor(scale, dtype=torch.float32)


def values(codes, scale):
    """Numbers of a cache [B, cap, H, d] in fp64."""
    return codes * np.repeat(scale, BLOCK, axis=1)[:, : codes.shape[1], :, None]


def decode(k, v, lengths, q, s=None, gain=None, tau=1.0):
    """k, v [B, cap, H, d] numbers, q [B, n_q, Hq, d]: (out, lse, weights [B, cap], sum of p |v|, logit scale)."""
    B, n_q, Hq, d = q.shape
    cap, H = k.shape[1], k.shape[2]
    out, lse = np.zeros((B, n_q, Hq, d)), np.full((B, n_q, Hq), -np.inf)
    mass, w, size = np.zeros((B, n_q, Hq, d)), np.zeros((B, cap)), 0.0
    for b in range(B):
        for i in range(n_q):
            n = lengths[b] - (n_q - 1 - i)
            if n <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[b, :n, h // (Hq // H)], v[b, :n, h // (Hq // H)]
                l = kk @ q[b, i, h] * (tau / math.sqrt(d))
                a = np.abs(kk) @ np.abs(q[b, i, h]) * abs(tau) / math.sqrt(d)
                if s is not None and gain is not None:
                    l = l + gain[h] * s[b, :n]
                    a = a + np.abs(np.where(np.isfinite(s[b, :n]), gain[h] * s[b, :n], 0.0))
                size = max(size, float(a.max()))
                m = l.max()
                if m == -np.inf:
                    continue
                p = np.exp(l - m)
                z = p.sum()
                p /= z
                lse[b, i, h] = m + math.log(z)
                out[b, i, h] = p @ np.where(p[:, None] > 0, vv, 0.0)
                mass[b, i, h] = p @ np.where(p[:, None] > 0, np.abs(vv), 0.0)
                w[b, :n] += p
    return out, lse, w, mass, size


def kept_slots(w, n, budget, sink, recent):
    if n <= budget:
        return list(range(n))
    mid = list(range(sink, n - recent))
    rank = lambda c: (0, -w[c], c) if w[c] == w[c] else (1, 0.0, c)  # noqa: E731
    return sorted(list(range(sink)) + sorted(mid, key=rank)[: budget - sink - recent] + list(range(n - recent, n)))
