"""Measured cases of the 8-bit decode cache: appending to it, attention over it, eviction from it.

A cache holds the keys and values of B sequences as 8-bit codes (e4m3 or int8), [B, capacity, Hkv, d],
with one scale, a power of two, for every block of 32 tokens and head, and per token a logit bias s
(the gate's score) and the attention weight w it has gathered so far.

`run` computes each operator in plain 32-bit torch operations, or, with `own`, calls the framework.
e4m3 codes are returned as float8 values beside their scales; int8 codes are read back as the values
they stand for.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32                                   # tokens under one scale
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------------------------------- cases
def _append(name, fmt, B, n_new, start, Hkv, d, ragged=False, fused=False):
    return {"name": name, "op": "append", "fmt": fmt, "B": B, "n_new": n_new, "start": start, "Hkv": Hkv, "d": d,
            "ragged": ragged, "fused": fused}


def _decode(name, fmt, B, T, Hq, Hkv, d, n_q=1, ragged=False, bias=True, weights=False):
    return {"name": name, "op": "decode", "fmt": fmt, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "d": d, "n_q": n_q,
            "ragged": ragged, "bias": bias, "weights": weights}


def _evict(name, fmt, B, T, budget, sink, recent, Hkv, d, ragged=False):
    return {"name": name, "op": "evict", "fmt": fmt, "B": B, "T": T, "budget": budget, "sink": sink, "recent": recent,
            "Hkv": Hkv, "d": d, "ragged": ragged}


def listed():
    return [
        # a decoding step's own key and value into the pruned 64k stack's cache (8704 kept tokens)
        _append("append 1 token", "e4m3", 1, 1, 8704, 8, 128),
        # the dense layers' prompt at 64k, keys and values as views of the projection's output
        _append("append 65536 tokens", "e4m3", 1, 65536, 0, 8, 128, fused=True),
        # a chunk of prompt for each of 16 sequences, of different lengths, into half-filled blocks; values read back
        _append("append ragged chunks", "int8", 16, 509, 331, 4, 128, ragged=True),
        # the small test stack's heads over a short cache: the launch's latency
        _decode("decode 257 keys", "e4m3", 1, 257, 4, 2, 64),
        # one step above the gate layer of the pruned 64k stack, gathering weights for a later eviction
        _decode("decode 8705 keys", "e4m3", 1, 8705, 16, 8, 128, weights=True),
        # one step of a dense layer at 64k
        _decode("decode 65537 keys", "e4m3", 1, 65537, 16, 8, 128, bias=False),
        # a batch of sequences of every length from none to 8705, 8 query heads to a key head
        _decode("decode ragged batch", "int8", 24, 8705, 32, 4, 128, ragged=True, weights=True),
        # four tokens of a draft checked at once
        _decode("decode 4 queries", "int8", 1, 32769, 16, 8, 128, n_q=4),
        # two sequences at 128k with the weights
        _decode("decode 131073 keys", "e4m3", 2, 131073, 16, 8, 128, weights=True),
        # the pruned stack's cache, grown by 257 tokens, cut back to what the gate had kept
        _evict("evict 8961 to 8704", "e4m3", 1, 8961, 8704, 4, 512, 8, 128),
        # a dense 64k cache cut to the pruned cache's size
        _evict("evict 65537 to 8704", "e4m3", 1, 65537, 8704, 4, 512, 8, 128),
        # a batch of different lengths, some shorter than the budget; values read back
        _evict("evict ragged batch", "int8", 12, 4099, 1024, 1, 63, 4, 128, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "decode", "decode", "evict"))
    fmt = rng.choice(("e4m3", "int8"))
    B = _log(rng, 1, 24)
    Hkv = rng.choice((1, 2, 4, 8))
    d = rng.choice((64, 128))
    most = max(2, min(131073, 65537 * 8 * 128 // (B * Hkv * d)))   # tokens a sequence may have
    ragged = B > 1 and rng.random() < 0.6
    if op == "append":
        n_new = _log(rng, 1, max(1, most // 2))
        return _append(None, fmt, B, n_new, rng.randrange(0, 1 + min(most // 4, 9000)), Hkv, d, ragged,
                       rng.random() < 0.5) | {"name": ""}
    T = _log(rng, 1, most)
    if op == "decode":
        G = rng.choice((1, 2, 3, 4, 8))
        n_q = rng.choice((1, 1, 1, 2, 16 // G))
        return _decode("", fmt, B, T, G * Hkv, Hkv, d, max(1, min(n_q, 16 // G)), ragged, rng.random() < 0.7,
                       rng.random() < 0.5)
    budget = _log(rng, 1, T)
    sink = rng.randrange(0, 1 + min(8, budget))
    return _evict("", fmt, B, T, budget, sink, rng.randrange(0, 1 + min(512, budget - sink)), Hkv, d, ragged)


def _spread(n, B, ragged):
    """Lengths of the B sequences: all n, or spread from none to n in a mixed order."""
    if not ragged or B == 1:
        return [n] * B
    return [n * ((b * 7 + 3) % B if B % 7 else b) // (B - 1) for b in range(B)]


def _capacity(n):
    return -(-n // BLOCK) * BLOCK + 2 * BLOCK


# ------------------------------------------------------------------------------------------- plain forms
def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _exponent(amax, fmt):
    """The least e >= -126 with amax <= qmax 2^e; -126 where amax is 0."""
    m, x = torch.frexp(amax)                  # amax = m 2^x, m in [1/2, 1)
    if fmt == "e4m3":                         # 448 = 0.875 * 2^9
        e = torch.where(m <= 0.875, x - 9, x - 8)
    else:                                     # 127 = 0.9921875 * 2^7
        e = torch.where(m <= 0.9921875, x - 7, x - 6)
    return torch.where(amax == 0, torch.full_like(e, -126), e.clamp(min=-126)).to(torch.int32)


def _codes(x, fmt):
    return x.to(CODE[fmt]) if fmt == "e4m3" else torch.round(x).to(torch.int8)


def _quantize(x, fmt):
    """x [B, T, H, d] fp32, T a multiple of 32: (codes, scales [B, T / 32, H])."""
    B, T, H, d = x.shape
    xb = x.view(B, T // BLOCK, BLOCK, H, d)
    scale = _pow2(_exponent(xb.abs().amax((2, 4)), fmt))
    return _codes(xb / scale[:, :, None, :, None], fmt).view(B, T, H, d), scale


def _values(codes, scale, T):
    """The fp32 values of the first T tokens."""
    B, _, H, d = codes.shape
    nb = -(-T // BLOCK)
    x = codes[:, : nb * BLOCK].float().view(B, nb, BLOCK, H, d) * scale[:, :nb, None, :, None]
    return x.view(B, nb * BLOCK, H, d)[:, :T]


def _append_plain(st, codes, scale, x):
    """x's rows to slots [length - count, length) of `codes`, the touched blocks' scales grown where needed."""
    B, n, H, d = x.shape
    fmt, dev = st["fmt"], x.device
    start = (st["lengths"] - st["counts"]).long()
    nblk = (n + BLOCK - 2) // BLOCK + 1
    blk = start[:, None] // BLOCK + torch.arange(nblk, device=dev)                       # [B, nblk]
    slot = (blk[:, :, None] * BLOCK + torch.arange(BLOCK, device=dev)).view(B, -1)       # [B, nblk * 32]
    row = slot - start[:, None]
    new = (row >= 0) & (row < st["counts"][:, None])
    old = row < 0
    bi = torch.arange(B, device=dev)[:, None]
    xn = x[bi, row.clamp(0, n - 1)].float() * new[:, :, None, None]
    s_old = scale[bi, blk]                                                               # [B, nblk, H]
    has_old = old.view(B, nblk, BLOCK).any(2)
    touched = new.view(B, nblk, BLOCK).any(2)
    s_new = _pow2(_exponent(xn.view(B, nblk, BLOCK, H, d).abs().amax((2, 4)), fmt))
    s_new = torch.where(has_old[:, :, None], torch.maximum(s_new, s_old), s_new)
    c_old = codes[bi, slot]
    ratio = (s_old / s_new).repeat_interleave(BLOCK, 1)[..., None]
    c_moved = _codes(c_old.float() * ratio, fmt)
    c_new = _codes(xn / s_new.repeat_interleave(BLOCK, 1)[..., None], fmt)
    live = touched.repeat_interleave(BLOCK, 1)
    as8 = lambda t: t.view(torch.uint8)  # noqa: E731
    c = torch.where((old & live)[:, :, None, None], as8(c_moved), torch.where(new[:, :, None, None], as8(c_new), as8(c_old)))
    as8(codes)[bi, slot] = c
    scale[bi, blk] = torch.where(touched[:, :, None], s_new, s_old)
    return slot, new, row


def _run_append(st):
    slot, new, row = _append_plain(st, st["k8"], st["k_scale"], st["k"])
    _append_plain(st, st["v8"], st["v_scale"], st["v"])
    B, n = st["s_new"].shape
    bi = torch.arange(B, device=slot.device)[:, None]
    st["s"][bi, slot] = torch.where(new, st["s_new"][bi, row.clamp(0, n - 1)], st["s"][bi, slot])
    st["w"][bi, slot] = torch.where(new, torch.zeros_like(st["s"][bi, slot]), st["w"][bi, slot])


def _run_decode(st):
    q, T, tau = st["q"].float(), st["T"], st["tau"]
    B, n_q, Hq, d = q.shape
    Hkv = st["k8"].shape[2]
    G = Hq // Hkv
    k, v = _values(st["k8"], st["k_scale"], T), _values(st["v8"], st["v_scale"], T)
    qh = q.view(B, n_q, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n_q * G, d)
    l = torch.matmul(qh, k.permute(0, 2, 3, 1)).view(B, Hkv, n_q, G, T) * (tau / math.sqrt(d))
    if st["s"] is not None:
        l = l + st["gain"].view(1, Hkv, 1, G, 1) * st["s"][:, None, None, None, :T]
    last = st["lengths"].view(B, 1) - (n_q - 1) + torch.arange(n_q, device=q.device)     # keys query i sees
    seen = torch.arange(T, device=q.device) < last[:, :, None]                           # [B, n_q, T]
    l = l.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    m = l.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(l - m)
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z == 0, torch.ones_like(z), z)
    v = v.masked_fill((torch.arange(T, device=q.device) >= st["lengths"][:, None])[:, :, None, None], 0.0)
    o = torch.matmul(p.view(B, Hkv, n_q * G, T), v.permute(0, 2, 1, 3)).view(B, Hkv, n_q, G, d)
    out = o.permute(0, 2, 1, 3, 4).reshape(B, n_q, Hq, d).to(torch.bfloat16)
    lse = (m + torch.log(z)).view(B, Hkv, n_q, G).permute(0, 2, 1, 3).reshape(B, n_q, Hq)
    if st["w"] is not None:
        st["w"][:, :T] += p.sum((1, 2, 3))
    return out, lse


def _run_evict(st):
    n, budget, sink, recent = st["lengths"].long()[:, None], st["budget"], st["sink"], st["recent"]
    B, cap = st["w"].shape
    c = torch.arange(cap, device=n.device)
    key = torch.where((c < sink) | (c >= n - recent), torch.full_like(st["w"], float("inf")), st["w"])
    key = torch.where(c < n, key, torch.full_like(key, float("-inf")))
    first = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
    first = torch.where(first < n, first, torch.full_like(first, cap))                   # nothing there
    kept = torch.sort(first, 1).values
    live = kept < cap
    at = kept.clamp(max=cap - 1)
    pad = st["dst_w"].shape[1] - budget
    bi = torch.arange(B, device=n.device)[:, None]
    lived = torch.nn.functional.pad(live, (0, pad))
    for x in ("k", "v"):
        rows = st[x + "8"][bi, at].float() * st[x + "_scale"][bi, at // BLOCK][..., None]
        rows = torch.nn.functional.pad(rows * live[:, :, None, None], (0, 0, 0, 0, 0, pad))
        codes, scale = _quantize(rows, st["fmt"])
        old = st["dst_" + x + "8"].view(torch.uint8)
        old.copy_(torch.where(lived[:, :, None, None], codes.view(torch.uint8), old))
        some = lived.view(B, -1, BLOCK).any(2)[:, :, None]
        st["dst_" + x + "_scale"].copy_(torch.where(some, scale, st["dst_" + x + "_scale"]))
    for x in ("s", "w"):
        st["dst_" + x][:, :budget] = torch.where(live, st[x][bi, at], st["dst_" + x][:, :budget])
    st["dst_lengths"].copy_(live.sum(1))
    st["kept"].copy_(torch.where(live, kept, torch.full_like(kept, -1)))


def _read_back(st, codes, scale, T, into, lengths):
    """The values of the first lengths[b] tokens as bf16 into `into` [B, T, Hkv, d]; other rows stay."""
    live = (torch.arange(T, device=codes.device) < lengths[:, None])[:, :, None, None]
    into.copy_(torch.where(live, _values(codes, scale, T).to(torch.bfloat16), into))


# ------------------------------------------------------------------------------------------- inputs
def _fill(g, B, T, H, d, dev, heavy=True):
    """Keys or values N(0, 1), some tokens three times as large, in bf16."""
    x = torch.randn(B, T, H, d, generator=g, device=dev)
    if heavy:
        x *= torch.where(torch.rand(B, T, 1, 1, generator=g, device=dev) < 0.03, 3.0, 1.0)
    return x.to(torch.bfloat16)


def _cache(g, case, cap, dev):
    st = {}
    for x in ("k", "v"):
        codes, scale = _quantize(_fill(g, case["B"], cap, case["Hkv"], case["d"], dev).float(), case["fmt"])
        st[x + "8"], st[x + "_scale"] = codes, scale
    return st


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    B, H, d, fmt = case["B"], case["Hkv"], case["d"], case["fmt"]
    op = case["op"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if op == "append":
        n, start = case["n_new"], case["start"]
        cap = _capacity(start + n)
        st = _cache(g, case, cap, dev)
        counts = _spread(n, B, case["ragged"])
        if case["fused"]:            # views of one projection output of 2 Hkv query and 2 Hkv key and value heads
            qkv = _fill(g, B, n, 4 * H, d, dev)
            st["k"], st["v"] = qkv[:, :, 2 * H: 3 * H], qkv[:, :, 3 * H:]
        else:
            st["k"], st["v"] = _fill(g, B, n, H, d, dev), _fill(g, B, n, H, d, dev)
        st["s_new"] = torch.randn(B, n, generator=g, device=dev)
        st["counts"] = ints(counts)
        st["lengths"] = ints([start + c for c in counts])
        st["s"] = torch.randn(B, cap, generator=g, device=dev)
        st["w"] = torch.rand(B, cap, generator=g, device=dev)
        st["T"] = start + n
        if fmt == "int8":
            st["k_out"] = torch.zeros(B, start + n, H, d, dtype=torch.bfloat16, device=dev)
            st["v_out"] = torch.zeros_like(st["k_out"])
    elif op == "decode":
        T = case["T"]
        cap = _capacity(T)
        st = _cache(g, case, cap, dev)
        st["T"], st["tau"] = T, 1.1
        st["lengths"] = ints(_spread(T, B, case["ragged"]))
        st["q"] = torch.randn(B, case["n_q"], case["Hq"], d, generator=g, device=dev).to(torch.bfloat16)
        st["gain"] = 2.0 * torch.rand(case["Hq"], generator=g, device=dev) if case["bias"] else None
        st["s"] = 0.6 * torch.randn(B, cap, generator=g, device=dev) if case["bias"] else None
        st["w"] = torch.rand(B, cap, generator=g, device=dev) if case["weights"] else None
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(B, case["n_q"], case["Hq"], device=dev)
    else:
        T, budget = case["T"], case["budget"]
        cap, dcap = _capacity(T), _capacity(budget)
        st = _cache(g, case, cap, dev)
        st |= {"T": T, "budget": budget, "sink": case["sink"], "recent": case["recent"]}
        st["lengths"] = ints(_spread(T, B, case["ragged"]))
        st["s"] = 0.6 * torch.randn(B, cap, generator=g, device=dev)
        # sums of softmax weights: a few tokens hold most of them
        st["w"] = torch.exp(3.0 * torch.randn(B, cap, generator=g, device=dev)) / T
        st["kept"] = torch.full((B, budget), -1, dtype=torch.int32, device=dev)
        st["dst_lengths"] = ints([0] * B)
        st["dst_s"] = torch.zeros(B, dcap, device=dev)
        st["dst_w"] = torch.zeros(B, dcap, device=dev)
        for x in ("k", "v"):
            st["dst_" + x + "8"] = torch.zeros(B, dcap, H, d, dtype=torch.uint8, device=dev).view(CODE[fmt])
            st["dst_" + x + "_scale"] = torch.ones(B, dcap // BLOCK, H, device=dev)
        if fmt == "int8":
            st["k_out"] = torch.zeros(B, budget, H, d, dtype=torch.bfloat16, device=dev)
            st["v_out"] = torch.zeros_like(st["k_out"])
    st["op"], st["fmt"] = op, fmt
    if own:                          # the handles that a program keeps over its cache's buffers
        from learned_token_pruning_tg_b200.cache import KVCacheQ8
        st["cache"] = KVCacheQ8.over(st["k8"], st["v8"], st["k_scale"], st["v_scale"], st["lengths"], s=st["s"],
                                     w=st["w"])
        if op == "evict":
            st["dst"] = KVCacheQ8.over(st["dst_k8"], st["dst_v8"], st["dst_k_scale"], st["dst_v_scale"],
                                       st["dst_lengths"], s=st["dst_s"], w=st["dst_w"])
    return st


# ------------------------------------------------------------------------------------------- a pass
def run(st):
    op, fmt = st["op"], st["fmt"]
    if op == "append":
        if own:
            st["cache"].append(st["k"], st["v"], s=st["s_new"], counts=st["counts"])
        else:
            _run_append(st)
        if fmt == "e4m3":
            return {"k": st["k8"], "v": st["v8"], "k_scale": st["k_scale"], "v_scale": st["v_scale"], "s": st["s"],
                    "w": st["w"]}
        if own:
            st["cache"].read(st["k_out"], st["v_out"])
        else:
            _read_back(st, st["k8"], st["k_scale"], st["T"], st["k_out"], st["lengths"])
            _read_back(st, st["v8"], st["v_scale"], st["T"], st["v_out"], st["lengths"])
        return {"k": st["k_out"], "v": st["v_out"], "k_scale": st["k_scale"], "v_scale": st["v_scale"], "s": st["s"],
                "w": st["w"]}
    if op == "decode":
        if own:
            st["cache"].decode(st["q"], st["out"], gain=st["gain"], tau=st["tau"], lse=st["lse"],
                               accumulate=st["w"] is not None, max_len=st["T"])
            out, lse = st["out"], st["lse"]
        else:
            out, lse = _run_decode(st)
        return {"out": out, "lse": lse, "w": st["w"]}
    if own:
        st["cache"].evict_into(st["dst"], st["budget"], sink=st["sink"], recent=st["recent"], kept=st["kept"],
                               max_len=st["T"])
    else:
        _run_evict(st)
    res = {"kept": st["kept"], "lengths": st["dst_lengths"], "s": st["dst_s"], "w": st["dst_w"],
           "k_scale": st["dst_k_scale"], "v_scale": st["dst_v_scale"]}
    if fmt == "e4m3":
        return res | {"k": st["dst_k8"], "v": st["dst_v8"]}
    if own:
        st["dst"].read(st["k_out"], st["v_out"])
    else:
        _read_back(st, st["dst_k8"], st["dst_k_scale"], st["budget"], st["k_out"], st["dst_lengths"])
        _read_back(st, st["dst_v8"], st["dst_v_scale"], st["budget"], st["v_out"], st["dst_lengths"])
    return res | {"k": st["k_out"], "v": st["v_out"]}


def work(case):
    B, H, d = case["B"], case["Hkv"], case["d"]
    row = 2 * H * d                                             # 8-bit bytes of one token's key and value
    sc = 8 * H / BLOCK                                          # its share of the scales
    if case["op"] == "append":
        counts = _spread(case["n_new"], B, case["ragged"])
        n = sum(counts)
        total = n * (row * 3 + sc + 12)
        if case["fmt"] == "int8":                               # the values of the whole sequences read back
            total += sum(case["start"] + c for c in counts) * (row * 3 + sc)
        return {"bytes": total, "flops": 2 * n * row}
    if case["op"] == "decode":
        lens = _spread(case["T"], B, case["ragged"])
        T = sum(lens)
        rows = B * case["n_q"] * case["Hq"]
        per_key = row + sc + (4 if case["bias"] else 0) + (8 if case["weights"] else 0)
        return {"bytes": T * per_key + rows * (4 * d + 4), "flops": 4 * T * case["n_q"] * case["Hq"] * d}
    lens = _spread(case["T"], B, case["ragged"])
    K = sum(min(n, case["budget"]) for n in lens)
    total = 4 * sum(lens) + K * (2 * row + 2 * sc + 16)
    if case["fmt"] == "int8":
        total += K * (row * 3 + sc)
    return {"bytes": total, "flops": 2 * K * row}


# ------------------------------------------------------------------------------------------- 64 bits
def _round64(x, fmt):
    """x (fp64, within the range) to the nearest code value, ties to even."""
    if fmt == "int8":
        return torch.round(x)
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6)
    step = torch.exp2(e - 3)                                    # 3 fraction bits, the least exponent -6
    return torch.round(x / step) * step


def _scale64(amax, fmt):
    """2^e for the least e with amax <= qmax 2^e (a float)."""
    if amax == 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(amax / QMAX[fmt]))
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    while e > -126 and amax <= QMAX[fmt] * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -126)


def _scales64(amax, fmt):
    a = amax.double().cpu().numpy()
    return torch.tensor(np.vectorize(lambda t: _scale64(float(t), fmt), otypes=[np.float64])(a), device=amax.device)


def _block64(codes, scale, b, j):
    """Values of block j of sequence b in fp64 [32, H, d]."""
    return codes[b, j * BLOCK: (j + 1) * BLOCK].double() * scale[b, j].double()[None, :, None]


def exact(case, seed):
    st = prepare(case, seed)
    fmt, B = case["fmt"], case["B"]
    lens = [int(n) for n in st["lengths"].cpu()]
    if case["op"] == "append":
        res = {}
        counts = [int(c) for c in st["counts"].cpu()]
        for x in ("k", "v"):
            codes, scale = st[x + "8"].double(), st[x + "_scale"].double()
            for b in range(B):
                if counts[b] == 0:
                    continue
                first, end = lens[b] - counts[b], lens[b]
                rows = st[x][b, :counts[b]].double()
                j0, j1 = first // BLOCK, (end - 1) // BLOCK + 1
                span = torch.zeros(j1 * BLOCK - j0 * BLOCK, *rows.shape[1:], dtype=torch.float64, device=rows.device)
                span[first - j0 * BLOCK: end - j0 * BLOCK] = rows
                sc = _scales64(span.view(j1 - j0, BLOCK, *rows.shape[1:]).abs().amax((1, 3)), fmt)   # [blocks, H]
                if first % BLOCK:
                    before = scale[b, j0].clone()
                    sc[0] = torch.maximum(sc[0], before)
                    resident = codes[b, j0 * BLOCK: first]
                    codes[b, j0 * BLOCK: first] = _round64(resident * (before / sc[0])[None, :, None], fmt)
                each = sc.repeat_interleave(BLOCK, 0)[first - j0 * BLOCK: end - j0 * BLOCK]
                codes[b, first:end] = _round64(rows / each[:, :, None], fmt)
                scale[b, j0:j1] = sc
            res[x], res[x + "_scale"] = codes, scale
            if fmt == "int8":
                values = codes[:, : st["T"]] * scale.repeat_interleave(BLOCK, 1)[:, : st["T"], :, None]
                for b in range(B):
                    values[b, lens[b]:] = 0.0
                res[x] = values
        s, w = st["s"].double(), st["w"].double()
        for b in range(B):
            s[b, lens[b] - counts[b]: lens[b]] = st["s_new"][b, :counts[b]].double()
            w[b, lens[b] - counts[b]: lens[b]] = 0.0
        return res | {"s": s, "w": w}
    if case["op"] == "decode":
        Hq, n_q, d, G = case["Hq"], case["n_q"], case["d"], case["Hq"] // case["Hkv"]
        out = torch.zeros(B, n_q, Hq, d, dtype=torch.float64, device=st["q"].device)
        lse = torch.full((B, n_q, Hq), float("-inf"), dtype=torch.float64, device=out.device)
        w = None if st["w"] is None else st["w"].double()
        for b in range(B):
            n = lens[b]
            for h in range(Hq):
                kv = h // G
                of = lambda c, sc: c[b, :n, kv].double() * sc[b, :, kv].double().repeat_interleave(BLOCK)[:n, None]  # noqa: E731
                if h % G == 0:
                    keys, vals = of(st["k8"], st["k_scale"]), of(st["v8"], st["v_scale"])
                for i in range(n_q):
                    m = n - (n_q - 1 - i)
                    if m <= 0:
                        continue
                    l = keys[:m] @ st["q"][b, i, h].double() * (st["tau"] / math.sqrt(d))
                    if st["s"] is not None:
                        l = l + float(st["gain"][h]) * st["s"][b, :m].double()
                    lse[b, i, h] = torch.logsumexp(l, 0)
                    p = torch.exp(l - lse[b, i, h])
                    out[b, i, h] = p @ vals[:m]
                    if w is not None:
                        w[b, :m] += p
        return {"out": out, "lse": lse, "w": w}
    budget, sink, recent = case["budget"], case["sink"], case["recent"]
    res = {"k": st["dst_k8"].double(), "v": st["dst_v8"].double(), "k_scale": st["dst_k_scale"].double(),
           "v_scale": st["dst_v_scale"].double(), "s": st["dst_s"].double(), "w": st["dst_w"].double()}
    kept_all = st["kept"].clone()
    new_lens = []
    for b in range(B):
        n = lens[b]
        w = st["w"][b, :n].double().cpu().numpy()
        if n <= budget:
            kept = np.arange(n)
        else:
            mid = np.arange(sink, n - recent)
            best = mid[np.lexsort((mid, -w[mid]))][: budget - sink - recent]
            kept = np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)]))
        K = len(kept)
        new_lens.append(K)
        at = torch.tensor(kept, dtype=torch.long, device=kept_all.device)
        kept_all[b, :K] = at.to(torch.int32)
        for x in ("s", "w"):
            res[x][b, :K] = st[x][b][at].double()
        for x in ("k", "v"):
            rows = st[x + "8"][b][at].double() * st[x + "_scale"][b][at // BLOCK].double()[:, :, None]
            nb = -(-K // BLOCK)
            if nb == 0:
                continue
            full = torch.zeros(nb * BLOCK, *rows.shape[1:], dtype=torch.float64, device=rows.device)
            full[:K] = rows
            sc = _scales64(full.view(nb, BLOCK, *rows.shape[1:]).abs().amax((1, 3)), fmt)
            res[x + "_scale"][b, :nb] = sc
            res[x][b, :K] = _round64(rows / sc.repeat_interleave(BLOCK, 0)[:K, :, None], fmt)
    if fmt == "int8":
        for x in ("k", "v"):
            res[x] = (res[x] * res[x + "_scale"].repeat_interleave(BLOCK, 1)[..., None])[:, :budget]
    return res | {"kept": kept_all, "lengths": torch.tensor(new_lens, dtype=torch.int32, device=kept_all.device)}
