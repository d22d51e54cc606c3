"""The 8-bit cache's kernels against the 64-bit reference (tests/cache_ref.py).

Appending, reading back and eviction are exact: scales are powers of two, so every code is one rounding of a number
that is exact on both sides, and the results are compared bit for bit.

Attention, with S = sum |q_i k_i| |tau| / sqrt(d) + |gain s| the size of a logit's terms: the products are exact in
fp32 (8 + 11 bits), and the tensor cores add d of them with at most d roundings of 2^-23 of the running magnitude; the
scaling, the bias and the difference to the maximum add a few more.  So a logit is off by at most
e = (d + 8) 2^-23 S, a weight by the factor exp(2 e) (its own and the sum's) plus ex2.approx (2^-22), P's
rounding to fp16 (2^-12, ten times less common in the mean, counted whole) and the sums' fp32 (2^-20 for the lengths
here).  Hence |out - want| <= (2 e + 2^-12 + 2^-19) sum_c p_c |v_c|, times 1 + 2^-8, and half a bf16 step of the
result (2^-9 of its power of two, 2^-8 relative at most); |lse - want| <= e + 2^-20 + 2^-23 |lse|; a
token's weight (2 e + 2^-18) of itself.  (Weights below 2^-18 of the reference are rounded in steps of 2^-28 of it: 2^17 keys
of such weights together would be 2^-12 off, the bound's own; these inputs leave few of them.)
"""
import numpy as np
import pytest
import torch

from learned_token_pruning_tg_b200 import tokengate as tg
from learned_token_pruning_tg_b200.cache import KVCacheQ8
from tests import cache_ref as ref
from tests.guards import guarded

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "int8"]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def guarded_cache(fmt, B, cap, H, d, bias=True, weights=True):
    """An empty cache whose code, scale and per-token buffers lie between guard bands."""
    checks = []

    def new(shape, dtype):
        t, check = guarded(shape, dtype)
        checks.append(check)
        return t

    k, v = (new((B, cap, H, d), torch.uint8) for _ in range(2))
    ks, vs = (new((B, cap // 32, H), torch.float32) for _ in range(2))
    k.fill_(0x7f)                       # NaN codes (int8: 127) where nothing was written
    v.fill_(0x7f)
    ks.fill_(float("nan"))
    vs.fill_(float("nan"))
    s = new((B, cap), torch.float32).fill_(float("nan")) if bias else None
    w = new((B, cap), torch.float32).fill_(float("nan")) if weights else None
    lengths = new((B,), torch.int32).zero_()
    c = KVCacheQ8.over(k.view(ref.DTYPE[fmt]), v.view(ref.DTYPE[fmt]), ks, vs, lengths, s=s, w=w)
    return c, lambda: [check() for check in checks]


def heavy(g, *shape):
    x = torch.randn(*shape, generator=g)
    x *= torch.where(torch.rand(shape[0], shape[1], 1, 1, generator=g) < 0.05, 8.0, 1.0)
    return x.to(torch.bfloat16)


def bits(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def codes_of(num, fmt):
    """Code bytes of reference numbers (the sign of a zero is the kernel's: compared as numbers)."""
    return torch.tensor(num).to(torch.float32).to(ref.DTYPE[fmt])


def same_numbers(t, want):
    got = ref.code_values(t)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


# ------------------------------------------------------------------------------------------- append and read
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,H,d,cap,steps", [
    (1, 1, 64, 32, [[1], [1], [1]]),                         # token by token
    (1, 8, 128, 64, [[33], [1], [30]]),                      # into half a block, one token, to the last slot
    (3, 2, 128, 96, [[0, 1, 65], [32, 0, 31], [64, 95, 0]]),  # ragged, none, exactly full
    (2, 3, 64, 128, [[31, 32], [1, 96], [96, 0]]),           # ends and begins on a block's border
    (5, 5, 128, 32, [[7, 0, 32, 1, 31], [25, 3, 0, 31, 1]]),
])
def test_append_and_read(fmt, B, H, d, cap, steps):
    g = torch.Generator().manual_seed(B * 100 + cap + d)
    cache, check = guarded_cache(fmt, B, cap, H, d)
    codes = {n: ref.code_values(t) for n, t in (("k", cache.k), ("v", cache.v))}
    scale = {n: t.double().cpu().numpy() for n, t in (("k", cache.k_scale), ("v", cache.v_scale))}
    lens = [0] * B
    s_want, w_want = np.full((B, cap), np.nan), np.full((B, cap), np.nan)
    for i, counts in enumerate(steps):
        n = max(counts)
        # magnitudes that grow by far from step to step, so that scales grow inside blocks
        x = {m: heavy(g, B, n, H, d) * (20.0 ** (i - 1)) for m in ("k", "v")}
        x = {m: t.to(torch.bfloat16) for m, t in x.items()}
        s = torch.randn(B, n, generator=g)
        lens = [a + c for a, c in zip(lens, counts)]
        cache.lengths.copy_(ints(lens))
        cache.append(x["k"].cuda(), x["v"].cuda(), s=s.cuda(),
                     counts=None if counts == [n] * B else ints(counts))
        for m in ("k", "v"):
            codes[m], scale[m] = ref.append(codes[m], scale[m], lens, counts, x[m].double().numpy(), fmt)
        for b in range(B):
            s_want[b, lens[b] - counts[b]: lens[b]] = s[b, :counts[b]]
            w_want[b, lens[b] - counts[b]: lens[b]] = 0.0
    torch.cuda.synchronize()
    check()
    assert cache.device_status() == 0
    for m, t, sc in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        same_numbers(t, codes[m])                           # rows behind the sequences too: as they were
        assert np.array_equal(sc.double().cpu().numpy(), scale[m], equal_nan=True)
    assert np.array_equal(cache.s.double().cpu().numpy(), s_want, equal_nan=True)
    assert np.array_equal(cache.w.double().cpu().numpy(), w_want, equal_nan=True)
    # read back, from the start and from the middle
    for first, n in ((0, cap), (5, cap - 9)):
        (ko, ck), (vo, cv) = (guarded((B, n, H, d), torch.bfloat16) for _ in range(2))
        ko.fill_(7.0)
        vo.fill_(7.0)
        cache.read(ko, vo, first=first)
        ck()
        cv()
        for out, m in ((ko, "k"), (vo, "v")):
            want = ref.values(codes[m], scale[m])[:, first: first + n]
            for b in range(B):
                want[b, max(0, lens[b] - first):] = 7.0
            assert np.array_equal(out.double().cpu().numpy(), want)


def test_append_long_and_strided():
    """Keys and values as views of one projection output, a long prompt (quantized by torch as well)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    B, n, H, d = 1, 5003, 8, 128
    qkv = torch.randn(B, n, 4 * H, d, generator=g, device="cuda").to(torch.bfloat16)
    k, v = qkv[:, :, 2 * H: 3 * H], qkv[:, :, 3 * H:]
    for fmt in FORMATS:
        cache = KVCacheQ8(B, n, H, d, fmt=fmt)
        cache.lengths.fill_(n)
        cache.append(k, v)
        for x, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
            pad = torch.nn.functional.pad(x.double(), (0, 0, 0, 0, 0, -n % 32)).view(B, -1, 32, H, d)
            amax = pad.abs().amax((2, 4))
            want = torch.exp2(torch.ceil(torch.log2(amax / ref.QMAX[fmt])))
            assert torch.equal(scale.double(), want)
            y = (pad / want[:, :, None, :, None]).view(B, -1, H, d)[:, :n].float()
            want_codes = y.to(torch.float8_e4m3fn).float() if fmt == "e4m3" else torch.round(y)
            assert torch.equal(codes[:, :n].float(), want_codes)
            assert bool((codes[:, n:].float() == 0).all())
        assert bool((cache.s == 0).all()) and cache.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_not_finite(fmt):
    cache, check = guarded_cache(fmt, 1, 32, 2, 64)
    x = torch.ones(1, 4, 2, 64, dtype=torch.bfloat16)
    x[0, 1, 0, 3], x[0, 2, 0, 5], x[0, 3, 0, 7] = float("inf"), float("-inf"), float("nan")
    cache.lengths.fill_(4)
    cache.append(x.cuda(), torch.ones_like(x).cuda())
    check()
    assert cache.device_status() == tg.TG_STATUS_CACHE_VALUE
    want, scale = ref.append(ref.code_values(cache.k) * 0 + 0.0, np.zeros((1, 1, 2)), [4], [4], x.double().numpy(), fmt)
    same_numbers(cache.k[:, :4], want[:, :4])
    top = ref.QMAX[fmt]
    assert want[0, 1, 0, 3] == top and want[0, 2, 0, 5] == -top
    assert np.isnan(want[0, 3, 0, 7]) if fmt == "e4m3" else want[0, 3, 0, 7] == 0
    assert np.array_equal(cache.k_scale.double().cpu().numpy(), scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_extremes(fmt):
    """The largest and smallest bf16 numbers, zeros, and a block of zeros that grows."""
    big = torch.finfo(torch.bfloat16).max
    for value in (big, 2.0 ** -126, 2.0 ** -133, 0.0, -big):
        cache, check = guarded_cache(fmt, 1, 32, 1, 64)
        x = torch.full((1, 3, 1, 64), value).to(torch.bfloat16)
        x[0, 1] = 0
        cache.lengths.fill_(3)
        cache.append(x.cuda(), x.cuda())
        codes, scale = ref.append(np.zeros((1, 32, 1, 64)), np.zeros((1, 1, 1)), [3], [3], x.double().numpy(), fmt)
        y = torch.randn(1, 2, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        cache.lengths.fill_(5)
        cache.append(y.cuda(), y.cuda())
        codes, scale = ref.append(codes, scale, [5], [2], y.double().numpy(), fmt)
        check()
        same_numbers(cache.v[:, :5], codes[:, :5])
        assert float(cache.v_scale) == scale[0, 0, 0] and cache.device_status() == 0


def test_append_bad_lengths_and_counts():
    """Tokens that would lie outside the cache are not written, and the status says so."""
    H, d = 2, 64
    for lengths, counts, slots in (([40, -3], [8, 2], ([(0, s) for s in range(0)])), ([33, 3], [2, 9], None),
                                   ([2, 1], [5, 0], None)):
        cache, check = guarded_cache("int8", 2, 32, H, d)
        before = cache.k.clone()
        x = torch.full((2, 8, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        cache.lengths.copy_(ints(lengths))
        cache.append(x, x, counts=ints(counts))
        check()
        assert cache.device_status() & tg.TG_STATUS_CACHE_LENGTH
        for b in range(2):
            c = min(max(counts[b], 0), 8)
            new = [t for t in range(lengths[b] - c, lengths[b]) if 0 <= t < 32]
            for t in range(32):
                if t in new:
                    assert bool((cache.k[b, t].float() * cache.k_scale[b, 0, 0] == 3.0).all()), (b, t)
                else:
                    assert torch.equal(cache.k[b, t], before[b, t]), (b, t)


# ------------------------------------------------------------------------------------------- attention
def random_cache(fmt, B, cap, H, d, lengths, seed, bias=True, pow2=True):
    """Codes of normal numbers under scales of their own per block; NaN codes, NaN scales and weights of NaN
    behind every sequence."""
    g = torch.Generator().manual_seed(seed)
    cache, check = guarded_cache(fmt, B, cap, H, d, bias=bias)
    lens = list(lengths)
    cache.lengths.copy_(ints(lens))
    nums = {}
    for m, t, sc in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        sigma = 100.0 if fmt == "e4m3" else 30.0
        x = (torch.randn(B, cap, H, d, generator=g) * sigma).clamp(-ref.QMAX[fmt], ref.QMAX[fmt])
        codes = x.to(torch.float8_e4m3fn) if fmt == "e4m3" else torch.round(x).to(torch.int8)
        e = torch.randint(-1, 2, (B, cap // 32, H), generator=g).float()
        scale = torch.exp2(e) / sigma if not pow2 else torch.exp2(e - (6 if fmt == "e4m3" else 5))
        for b in range(B):
            codes.view(torch.uint8)[b, lens[b]:] = 0x7f
            scale[b, -(-lens[b] // 32):] = float("nan")
        t.copy_(codes)
        sc.copy_(scale)
        nums[m] = ref.values(np.nan_to_num(ref.code_values(codes)), np.nan_to_num(scale.double().numpy()))
    s = None
    if bias:
        s = torch.randn(B, cap, generator=g)
        for b in range(B):
            s[b, lens[b]:] = float("nan")
        cache.s.copy_(s)
    w = torch.rand(B, cap, generator=g)
    cache.w.copy_(w)
    return cache, check, nums, s, w, g


def half_step(x):
    a = np.abs(x)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    return np.where(a > 0, 2.0 ** (e - 8), 0.0)


def check_decode(cache, check, nums, s, w, q, gain, tau, lens, accumulate=True, max_len=0):
    B, n_q, Hq, d = q.shape
    out, co = guarded((B, n_q, Hq, d), torch.bfloat16)
    lse, cl = guarded((B, n_q, Hq), torch.float32)
    out.fill_(float("nan"))
    lse.fill_(float("nan"))
    cache.decode(q.cuda(), out, gain=None if gain is None else gain.cuda(), tau=tau, lse=lse, accumulate=accumulate,
                 max_len=max_len)
    torch.cuda.synchronize()
    for c in (check, co, cl):
        c()
    assert cache.device_status() == 0
    want, want_lse, want_w, mass, size = ref.decode(
        nums["k"], nums["v"], lens, q.double().numpy(), None if s is None else s.double().numpy(),
        None if gain is None else gain.double().numpy(), tau)
    e = (d + 8) * 2.0 ** -23 * size
    got = out.double().cpu().numpy()
    bound = (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(want) + 2.0 ** -10 * mass)
    assert np.all(np.abs(got - want) <= bound), np.max(np.abs(got - want) - bound)
    gl = lse.double().cpu().numpy()
    seen = np.isfinite(want_lse)
    assert np.array_equal(np.isfinite(gl), seen) and np.all(gl[~seen] == -np.inf)
    if seen.any():
        assert np.all(np.abs(gl[seen] - want_lse[seen]) <= e + 2.0 ** -20 + 2.0 ** -23 * np.abs(want_lse[seen]))
    gw = cache.w.double().cpu().numpy()
    w0 = w.double().numpy()
    for b in range(B):
        n = lens[b]
        if accumulate:
            tol = (2 * e + 2.0 ** -18) * want_w[b, :n] + 2.0 ** -23 * (w0[b, :n] + want_w[b, :n])
            assert np.all(np.abs(gw[b, :n] - w0[b, :n] - want_w[b, :n]) <= tol)
        else:
            assert np.array_equal(gw[b, :n], w0[b, :n])
        assert np.array_equal(gw[b, n:], w0[b, n:])         # nothing behind the sequence changes
    return out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,lens,Hq,Hkv,d,n_q", [
    (1, [1], 2, 1, 128, 1),
    (1, [0], 4, 2, 64, 1),                                  # no token at all
    (1, [31], 4, 2, 64, 1),
    (1, [33], 16, 8, 128, 1),
    (1, [1000], 3, 1, 64, 1),                               # 3 query heads a KV head
    (1, [2049], 32, 4, 128, 1),                             # G = 8
    (1, [777], 16, 1, 128, 1),                              # G = 16
    (4, [0, 1, 32, 300], 8, 8, 64, 1),                      # G = 1, ragged
    (7, [5, 0, 0, 257, 64, 1, 96], 10, 2, 128, 1),          # G = 5
    (2, [3, 130], 4, 2, 64, 4),                             # more queries than tokens: rows that see none
    (3, [0, 1, 513], 6, 2, 128, 5),                         # 15 rows a KV head, rows empty
    (1, [1024], 16, 8, 128, 8),                             # 16 rows
    (140, [i % 37 for i in range(140)], 4, 2, 64, 2),       # more sequences than threads of a block
])
def test_decode_parity(fmt, B, lens, Hq, Hkv, d, n_q):
    cap = (max(lens) + 32) // 32 * 32 + 32
    cache, check, nums, s, w, g = random_cache(fmt, B, cap, Hkv, d, lens, seed=sum(lens) + Hq + n_q)
    q = torch.randn(B, n_q, Hq, d, generator=g).to(torch.bfloat16)
    gain = 2 * torch.rand(Hq, generator=g)
    check_decode(cache, check, nums, s, w, q, gain, 1.3, lens)


def spread(n, most, seed):
    """n lengths between none and `most`, with runs of empty sequences."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, most + 1, (n,), generator=g)
    x[torch.rand(n, generator=g) < 0.2] = 0
    x[n // 3: n // 3 + 3] = 0
    x[n // 2] = most
    return x.tolist()


@pytest.mark.parametrize("fmt,B,most,Hq,Hkv,d,n_q", [
    ("e4m3", 40, 1100, 4, 2, 64, 1),       # more heads than clusters: equal runs over ragged sequences
    ("int8", 10, 1500, 24, 8, 128, 1),
    ("int8", 25, 1300, 12, 4, 64, 4),      # 12 rows a head
    ("e4m3", 400, 850, 1, 1, 64, 1),       # more sequences than threads of a block
])
def test_decode_ragged_runs(fmt, B, most, Hq, Hkv, d, n_q):
    lens = spread(B, most, B)
    cap = (most + 31) // 32 * 32
    cache, check, nums, s, w, g = random_cache(fmt, B, cap, Hkv, d, lens, seed=B + most)
    q = torch.randn(B, n_q, Hq, d, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, 2 * torch.rand(Hq, generator=g), 1.1, lens)


@pytest.mark.parametrize("max_len", [1, 400, 800, 1600, 3100, 6200, 0])
def test_decode_any_launch(max_len):
    """One thread block a head, a cluster of them, or runs: every launch reads the same caches whole."""
    lens = [13000, 0, 77]
    cache, check, nums, s, w, g = random_cache("e4m3", 3, 13024, 1, 64, lens, seed=21)
    q = torch.randn(3, 2, 3, 64, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, 2 * torch.rand(3, generator=g), 1.1, lens, max_len=max_len)


@pytest.mark.parametrize("Hq,d", [(3, 64), (5, 128), (15, 64)])
@pytest.mark.parametrize("T", [800, 1700, 2600, 3500, 4900, 6100])
def test_decode_any_cluster(T, Hq, d):
    """One KV head whose units go to 3 to 16 thread blocks, with rows that they do not share evenly."""
    cache, check, nums, s, w, g = random_cache("e4m3", 1, 6112, 1, d, [T], seed=T)
    q = torch.randn(1, 1, Hq, d, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, torch.rand(Hq, generator=g) * 2, 1.5, [T], max_len=T)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_without_bias_or_weights_and_any_scale(fmt):
    lens = [300, 45]
    cache, check, nums, s, w, g = random_cache(fmt, 2, 320, 2, 128, lens, seed=5, bias=False, pow2=False)
    q = torch.randn(2, 1, 4, 128, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, None, w, q, None, 0.7, lens, accumulate=False)
    cache, check, nums, s, w, g = random_cache(fmt, 2, 320, 2, 128, lens, seed=6)
    check_decode(cache, check, nums, None, w, q, None, -1.0, lens)       # no gain: no bias
    # a launch sized for shorter sequences than there are reads them whole all the same
    cache, check, nums, s, w, g = random_cache(fmt, 2, 320, 2, 128, lens, seed=7)
    check_decode(cache, check, nums, s, w, q, torch.ones(4), 1.0, lens, max_len=1)


@pytest.mark.parametrize("fmt", FORMATS)
def test_decode_masked_keys(fmt):
    """Biases of -inf and of the type's lowest value mask keys; a sequence whose keys are all masked gives 0."""
    lens = [100, 64, 65]
    cache, check, nums, s, w, g = random_cache(fmt, 3, 128, 2, 64, lens, seed=11)
    s[0, ::2] = float("-inf")
    s[1, :64] = float("-inf")
    s[2, 1:65] = torch.finfo(torch.float32).min             # times a gain above 1 that is -inf
    cache.s.copy_(s)
    q = torch.randn(3, 1, 4, 64, generator=g).to(torch.bfloat16)
    out, lse = check_decode(cache, check, nums, s, w, q, torch.full((4,), 1.5), 1.0, lens)
    assert bool((out[1] == 0).all()) and bool((lse[1] == float("-inf")).all())


@pytest.mark.parametrize("Hq,n_q", [(3, 1), (3, 5), (5, 3)])
def test_decode_odd_rows_with_masked_keys(Hq, n_q):
    """An odd number of rows a KV head: the row that pads the logits adds no weight, whatever the biases are."""
    lens = [70]
    cache, check, nums, s, w, g = random_cache("e4m3", 1, 96, 1, 64, lens, seed=15)
    s[0, 3:70:4] = float("-inf")
    cache.s.copy_(s)
    q = torch.randn(1, n_q, Hq, 64, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, torch.linspace(0.5, 1.5, Hq), 1.0, lens)


def test_decode_nan_and_inf_inputs():
    """What the formula makes of them: a NaN key or query gives NaN rows, and only those."""
    lens = [64, 64]
    cache, check, nums, s, w, g = random_cache("e4m3", 2, 64, 2, 64, lens, seed=12)
    cache.k.view(torch.uint8)[0, 5, 1, 3] = 0x7f            # NaN in sequence 0, KV head 1
    q = torch.randn(2, 1, 4, 64, generator=g).to(torch.bfloat16)
    q[1, 0, 2, 7] = float("nan")
    out = cache.decode(q.cuda(), gain=torch.ones(4, device="cuda"))
    bad = torch.isnan(out.float()).all(-1).cpu()[:, 0]
    some = torch.isnan(out.float()).any(-1).cpu()[:, 0]
    want = torch.tensor([[False, False, True, True], [False, False, True, False]])
    assert torch.equal(bad, want) and torch.equal(some, want)


def test_decode_large_and_small_magnitudes():
    """Queries far from 1 keep their bits (scaled by a power of two), and blocks of very different scales add up."""
    lens = [200]
    for mag in (2.0 ** 60, 2.0 ** -60):
        cache, check, nums, s, w, g = random_cache("int8", 1, 224, 2, 128, lens, seed=13, bias=False)
        q = (torch.randn(1, 1, 4, 128, generator=g) * mag).to(torch.bfloat16)
        check_decode(cache, check, nums, None, w, q, None, 1.0 / mag, lens)
    cache, check, nums, s, w, g = random_cache("e4m3", 1, 224, 2, 128, lens, seed=14)
    e = torch.tensor([-40.0, 0.0, 12.0, -3.0, -20.0, 7.0, -60.0])
    cache.v_scale.copy_(torch.exp2(e)[None, :, None].expand(1, 7, 2))
    nums["v"] = ref.values(np.nan_to_num(ref.code_values(cache.v)), cache.v_scale.double().cpu().numpy())
    q = torch.randn(1, 1, 4, 128, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, torch.ones(4), 1.0, lens)


def decode_in_torch(cache, q, gain, tau, lens):
    """fp64 on the device, for long caches (equal lengths)."""
    B, n_q, Hq, d = q.shape
    H, n = cache.Hkv, lens
    k, v = ((c[:, :n].double() * sc.double().repeat_interleave(32, 1)[:, :n, :, None])
            for c, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    qh = q.double().view(B, n_q, H, Hq // H, d)
    l = torch.einsum("bihgd,bchd->bihgc", qh, k) * (tau / d ** 0.5)
    size = torch.einsum("bihgd,bchd->bihgc", qh.abs(), k.abs()).max().item() * tau / d ** 0.5
    l = l + gain.double().view(H, -1, 1) * cache.s[:, None, None, None, :n].double()
    seen = torch.arange(n, device=q.device) < (n - (n_q - 1) + torch.arange(n_q, device=q.device))[:, None]
    l = l.masked_fill(~seen[:, None, None, :], float("-inf"))
    lse = torch.logsumexp(l, -1)
    p = torch.exp(l - lse[..., None])
    out = torch.einsum("bihgc,bchd->bihgd", p, v).reshape(B, n_q, Hq, d)
    mass = torch.einsum("bihgc,bchd->bihgd", p, v.abs()).reshape(B, n_q, Hq, d)
    return out, lse.view(B, n_q, Hq), p.sum((1, 2, 3)), mass, size


@pytest.mark.parametrize("fmt,T,Hq,Hkv,n_q", [("e4m3", 65537, 16, 8, 1), ("int8", 40001, 32, 4, 2),
                                              ("e4m3", 131073, 8, 1, 1)])
def test_decode_long(fmt, T, Hq, Hkv, n_q):
    d = 128
    g = torch.Generator(device="cuda").manual_seed(T)
    cache = KVCacheQ8(1, T, Hkv, d, fmt=fmt)
    cache.lengths.fill_(T)
    k, v = (torch.randn(1, T, Hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    cache.append(k, v, s=0.6 * torch.randn(1, T, generator=g, device="cuda"))
    q = torch.randn(1, n_q, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    gain = 2 * torch.rand(Hq, generator=g, device="cuda")
    lse = torch.empty(1, n_q, Hq, device="cuda")
    out = cache.decode(q, gain=gain, tau=1.2, lse=lse, accumulate=True)
    want, want_lse, want_w, mass, size = decode_in_torch(cache, q, gain, 1.2, T)
    assert cache.device_status() == 0
    e = (d + 8) * 2.0 ** -23 * (size + 4 * 0.6 * 5)
    err = (out.double() - want).abs()
    step = torch.exp2(torch.floor(torch.log2(want.abs() + 2.0 ** -10 * mass)) - 8)
    assert bool((err <= (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + step).all())
    assert float((lse.double() - want_lse).abs().max()) <= e + 2.0 ** -20 + 2.0 ** -23 * float(want_lse.abs().max())
    dw = (cache.w[:, :T].double() - want_w).abs()
    assert bool((dw <= (2 * e + 2.0 ** -18 + 2.0 ** -22) * want_w).all())
    # the same bits again (the weights have moved on, nothing else)
    again = cache.decode(q, gain=gain, tau=1.2, accumulate=True)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_offsets_past_32_bits():
    """The end of the second of two sequences of 2.2 million tokens, 4.5 GB into the codes, against a small cache with the
    same tokens at the same place of their blocks."""
    B, H, d, cap, n, new_ = 2, 8, 128, 2_200_000, 2_199_990, 70
    at = (n - new_) % 32
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(3, B, new_, H, d, generator=g, device="cuda").to(torch.bfloat16)
    bias = 0.6 * torch.randn(B, new_, generator=g, device="cuda")
    gain = 0.5 + torch.rand(2 * H, generator=g, device="cuda")
    q = torch.randn(B, 1, 2 * H, d, generator=g, device="cuda").to(torch.bfloat16)
    got = []
    for size, length in ((cap, n), (96, at + new_)):
        cache = KVCacheQ8(B, size, H, d)
        cache.k_scale.fill_(1.0)
        cache.v_scale.fill_(1.0)
        cache.s.fill_(float("-inf"))
        cache.lengths.copy_(ints([at + new_, length]))
        cache.append(x[0], x[1], bias)
        k, v = torch.empty_like(x[0]), torch.empty_like(x[1])
        cache.read(k, v, first=length - new_)
        lse = torch.empty(B, 1, 2 * H, device="cuda")
        out = cache.decode(q, gain=gain, tau=1.2, lse=lse, accumulate=True)
        dst = KVCacheQ8(B, new_, H, d)
        kept = cache.evict_into(dst, new_, recent=new_)
        assert torch.equal(kept[1], torch.arange(length - new_, length, dtype=torch.int32, device="cuda"))
        assert cache.device_status() == 0
        got.append((cache, k[1], v[1], out, lse, dst, cache.w[1, length - new_ : length].clone()))
    (_, k, v, out, lse, dst, w), (small, k2, v2, _, _, dst2, _) = got
    assert torch.equal(k, k2) and torch.equal(v, v2)
    for t, t2 in ((dst.k, dst2.k), (dst.v, dst2.v)):
        assert torch.equal(t[1, :new_].view(torch.uint8), t2[1, :new_].view(torch.uint8))
    assert torch.equal(dst.k_scale, dst2.k_scale) and torch.equal(dst.v_scale, dst2.v_scale)
    # the bounds of test_decode_long
    want, want_lse, want_w, mass, size = decode_in_torch(small, q, gain, 1.2, at + new_)
    e = (d + 8) * 2.0 ** -23 * (size + 4 * 0.6 * 5)
    err = (out.double() - want).abs()
    step = torch.exp2(torch.floor(torch.log2(want.abs() + 2.0 ** -10 * mass)) - 8)
    assert bool((err <= (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + step).all())
    assert float((lse.double() - want_lse).abs().max()) <= e + 2.0 ** -20 + 2.0 ** -23 * float(want_lse.abs().max())
    dw = (w.double() - want_w[1, at:]).abs()
    assert bool((dw <= (2 * e + 2.0 ** -18 + 2.0 ** -22) * want_w[1, at:]).all())


# ------------------------------------------------------------------------------------------- a step, captured
def test_steps_in_a_graph_and_on_streams():
    """Append and decode captured once and replayed while the sequences grow: the same bits as the calls made one by
    one on a stream of their own, and as a second graph over another cache, replayed at the same time."""
    B, H, Hq, d, start, steps = 3, 2, 4, 64, 700, 70      # from one thread block a head into clusters
    g = torch.Generator(device="cuda").manual_seed(9)
    first = torch.randn(2, B, start, H, d, generator=g, device="cuda").to(torch.bfloat16)
    news = torch.randn(steps, 3, B, 1, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    bias = torch.randn(steps, B, 1, generator=g, device="cuda")
    gain = torch.rand(Hq, generator=g, device="cuda")
    lens0 = ints([start, 0, start - 33])

    def fresh():
        c = KVCacheQ8(B, start + steps, H, d, fmt="e4m3")
        c.lengths.copy_(lens0)
        c.append(first[0], first[1], counts=lens0.clone())
        c.reserve(1, Hq, True)
        return c

    def step(c, q, k, v, s, out, lse):
        c.lengths.add_(1)
        c.append(k, v, s=s)
        c.decode(q, out, gain=gain, tau=1.2, lse=lse, accumulate=True)

    eager = fresh()
    want = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(steps):
            out, lse = torch.empty(B, 1, Hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(B, 1, Hq, device="cuda")
            step(eager, news[i, 0], news[i, 1][:, :, :H], news[i, 2][:, :, :H], bias[i], out, lse)
            want.append((out, lse))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        c = fresh()
        q = torch.empty(B, 1, Hq, d, dtype=torch.bfloat16, device="cuda")
        k, v = (torch.empty(B, 1, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        s, lse = torch.empty(B, 1, device="cuda"), torch.empty(B, 1, Hq, device="cuda")
        out = torch.empty_like(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(c, q, k, v, s, out, lse)
        graphs.append((graph, c, q, k, v, s, out, lse, torch.cuda.Stream()))
    for i in range(steps):
        for graph, c, q, k, v, s, out, lse, stream in graphs:
            with torch.cuda.stream(stream):
                q.copy_(news[i, 0])
                k.copy_(news[i, 1][:, :, :H])
                v.copy_(news[i, 2][:, :, :H])
                s.copy_(bias[i])
                graph.replay()
        torch.cuda.synchronize()
        for graph, c, q, k, v, s, out, lse, stream in graphs:
            assert torch.equal(out.view(torch.int16), want[i][0].view(torch.int16)), i
            assert torch.equal(lse, want[i][1]), i
    for graph, c, *_ in graphs:
        for name in ("k", "v", "k_scale", "v_scale", "s", "w", "lengths"):
            assert np.array_equal(bits(getattr(c, name)), bits(getattr(eager, name))), name
        assert c.device_status() == 0


def test_reserve_before_capture():
    cache = KVCacheQ8(1, 64, 1, 64)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="reserve"):
        with torch.cuda.graph(graph):
            cache.decode(q, out)
    torch.cuda.synchronize()
    assert bool((cache.decode(q, out) == 0).all())


def test_refusals_of_tensors():
    cache = KVCacheQ8(2, 64, 2, 64)
    new = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    x = new(2, 1, 2, 64)
    for bad in (new(2, 1, 2, 64, dt=torch.float16), x.cpu()):
        with pytest.raises(TypeError):
            cache.append(bad, x)
        with pytest.raises(TypeError):
            cache.decode(bad, out=new(2, 1, 2, 64))
    for bad in (new(1, 1, 2, 64), new(2, 1, 1, 64), new(2, 1, 2, 128), new(2, 1, 64, 2).transpose(2, 3)):
        with pytest.raises(ValueError):
            cache.append(bad, bad)
    with pytest.raises(ValueError):
        cache.append(x, new(2, 2, 2, 64))
    with pytest.raises(ValueError):
        cache.append(x, x, s=torch.zeros(2, 2, device="cuda"))
    with pytest.raises(TypeError):
        cache.append(x, x, counts=torch.ones(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        KVCacheQ8(2, 64, 2, 64, bias=False).append(x, x, s=torch.zeros(2, 1, device="cuda"))
    with pytest.raises(tg.TokenGateError):
        KVCacheQ8(2, 64, 2, 64, weights=False).decode(x, accumulate=True)
    for q in (new(2, 1, 3, 64), new(2, 9, 4, 64)):           # heads, rows a KV head
        with pytest.raises(tg.TokenGateError):
            cache.decode(q)
    with pytest.raises(ValueError):
        cache.decode(x, out=new(2, 1, 4, 64))
    with pytest.raises(ValueError):
        cache.decode(x, gain=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        cache.read(new(2, 3, 2, 64), new(2, 4, 2, 64))
    with pytest.raises(tg.TokenGateError):
        cache.read(new(2, 3, 2, 64), new(2, 3, 2, 64), first=62)
    with pytest.raises(tg.TokenGateError):
        cache.evict_into(cache, 32)                          # into itself
    with pytest.raises(tg.TokenGateError):
        cache.evict_into(KVCacheQ8(2, 32, 2, 64), 32, sink=20, recent=20)
    with pytest.raises(tg.TokenGateError):
        cache.evict_into(KVCacheQ8(2, 32, 2, 64, fmt="int8"), 32)
    base = new(2, 64, 2, 65, dt=torch.int8)[..., :64]
    with pytest.raises(ValueError, match="dense"):
        KVCacheQ8.over(base, base, torch.ones(2, 2, 2, device="cuda"), torch.ones(2, 2, 2, device="cuda"), ints([0, 0]))


def test_strided_cache():
    """K and V as views of one buffer (tokens of K and V codes side by side), sequences with room between them."""
    B, cap, H, d = 2, 64, 2, 64
    g = torch.Generator().manual_seed(4)
    buf = torch.full((B, cap + 32, 2, H, d), 0x7f, dtype=torch.uint8, device="cuda")
    k, v = (buf[:, :cap, i].view(torch.int8) for i in range(2))
    lens = [50, 64]
    cache = KVCacheQ8.over(k, v, torch.zeros(B, 2, H, device="cuda"), torch.zeros(B, 2, H, device="cuda"), ints(lens),
                           w=torch.zeros(B, cap, device="cuda"))
    x = torch.randn(2, B, 64, H, d, generator=g).to(torch.bfloat16)
    cache.append(x[0].cuda(), x[1].cuda(), counts=ints(lens))
    q = torch.randn(B, 1, 4, d, generator=g).to(torch.bfloat16)
    nums = {m: ref.values(ref.code_values(t), sc.double().cpu().numpy())
            for m, t, sc in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale))}
    check_decode(cache, lambda: None, nums, None, torch.zeros(B, cap), q, None, 1.0, lens)
    dst = KVCacheQ8(B, 32, H, d, fmt="int8")
    kept = cache.evict_into(dst, 20, sink=1, recent=2)
    for b in range(B):
        want, scale = ref.append(np.zeros((1, 32, H, d)), np.ones((1, 1, H)), [20], [20],
                                 nums["v"][b: b + 1, kept[b].tolist()], "int8")
        same_numbers(dst.v[b: b + 1], want)
    assert bool((buf[:, cap:] == 0x7f).all()) and bool((buf[0, 50:cap] == 0x7f).all())
    assert bool((dst.s[:, :20] == 0).all())


# ------------------------------------------------------------------------------------------- eviction
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,budget,sink,recent,H,d,wts", [
    ([100], 40, 4, 8, 2, 64, "random"),
    ([100], 40, 0, 0, 1, 128, "ties"),                      # many equal weights: the lower slots stay
    ([64], 33, 16, 17, 2, 64, "random"),                    # only protected tokens stay
    ([7, 0, 33, 96], 33, 1, 2, 3, 128, "special"),          # shorter, empty, equal, longer; NaN, infinities, -0
    ([50], 0, 0, 0, 1, 64, "random"),                       # nothing stays
    ([1], 1, 0, 1, 1, 64, "random"),
    ([96, 95], 95, 3, 5, 2, 64, "constant"),                # one token leaves
    ([3000, 2999], 1000, 4, 64, 1, 64, "random"),
    ([3000], 1000, 4, 64, 1, 64, "close"),                  # one first digit for all: every pass has to look
    ([3000], 1000, 4, 64, 1, 64, "two"),                    # two values, the budget between them
])
def test_evict(fmt, lens, budget, sink, recent, H, d, wts):
    B, cap = len(lens), (max(lens) + 31) // 32 * 32
    src, check, nums, s, w, g = random_cache(fmt, B, cap, H, d, lens, seed=cap + budget + sink)
    if wts == "ties":
        w = torch.randint(0, 4, (B, cap), generator=g).float()
    elif wts == "constant":
        w.fill_(0.25)
    elif wts == "close":
        w = 1.0 + torch.rand(B, cap, generator=g) * 2.0 ** -8
    elif wts == "two":
        w = torch.where(torch.arange(cap) % 3 == 0, 1.0, 0.5).expand(B, cap).contiguous()
    elif wts == "special":
        w = torch.randn(B, cap, generator=g)
        for i, x in enumerate((float("nan"), float("inf"), float("-inf"), 0.0, -0.0)):
            w[:, 5 + 3 * i::17] = x
    src.w.copy_(w)
    dst, check_dst = guarded_cache(fmt, B, (budget + 31) // 32 * 32 + 32, H, d)
    before = {n: getattr(dst, n).clone() for n in ("k", "v", "k_scale", "v_scale", "s", "w")}
    kept, ck = guarded((B, budget), torch.int32)
    src_before = bits(src.k).copy()
    src.evict_into(dst, budget, sink=sink, recent=recent, kept=kept)
    torch.cuda.synchronize()
    for c in (check, check_dst, ck):
        c()
    assert src.device_status() == 0 and np.array_equal(bits(src.k), src_before)
    got = kept.cpu().numpy()
    new = [min(n, budget) for n in lens]
    assert dst.lengths.cpu().tolist() == new
    for b in range(B):
        slots = ref.kept_slots(w[b].tolist(), lens[b], budget, sink, recent)
        assert got[b].tolist() == slots + [-1] * (budget - new[b])
        n = new[b]
        for name, ours in (("s", s), ("w", w)):
            have = getattr(dst, name)[b].cpu()
            assert np.array_equal(have[:n].numpy(), ours[b][slots].numpy(), equal_nan=True)
            assert np.array_equal(have[n:].numpy(), before[name][b, n:].cpu().numpy(), equal_nan=True)
        for m in ("k", "v"):
            codes = ref.code_values(before[m][b: b + 1])
            scale = before[m + "_scale"][b: b + 1].double().cpu().numpy()
            codes, scale = ref.append(codes, scale, [n], [n], nums[m][b: b + 1, slots], fmt)
            same_numbers(getattr(dst, m)[b: b + 1], codes)
            assert np.array_equal(getattr(dst, m + "_scale")[b: b + 1].double().cpu().numpy(), scale, equal_nan=True)


@pytest.mark.parametrize("T,budget,max_len", [(70001, 8704, 0), (70001, 8704, 1000), (450000, 20000, 0),
                                              (24000, 23000, 0), (30000, 29000, 0), (30000, 600, 0)])
def test_evict_long(T, budget, max_len):
    """Long sequences (keys in shared memory, or read again where they do not fit it or max_len was too small)."""
    g = torch.Generator(device="cuda").manual_seed(T)
    src = KVCacheQ8(1, T, 1, 64, fmt="int8", bias=False)
    src.lengths.fill_(T)
    x = torch.randn(1, T, 1, 64, generator=g, device="cuda").to(torch.bfloat16)
    src.append(x, x)
    src.w.copy_(torch.exp(3 * torch.randn(src.w.shape, generator=g, device="cuda")))
    src.w[:, 17::5] = 0.0                                   # long ties at the bottom
    dst = KVCacheQ8(1, budget, 1, 64, fmt="int8", bias=False)
    kept = src.evict_into(dst, budget, sink=4, recent=512, max_len=max_len)
    w = src.w[0, :T].cpu().numpy()
    mid = np.arange(4, T - 512)
    best = mid[np.lexsort((mid, -w[mid]))][: budget - 516]
    want = np.sort(np.concatenate([np.arange(4), best, np.arange(T - 512, T)]))
    assert np.array_equal(kept[0].cpu().numpy(), want)
    assert torch.equal(dst.w[0, :budget].cpu(), src.w[0].cpu()[want])


def test_evict_bad_length():
    src, check, nums, s, w, g = random_cache("int8", 2, 64, 1, 64, [64, 64], seed=3)
    src.lengths.copy_(ints([80, -5]))                       # clamped to 64 and 0
    dst, check_dst = guarded_cache("int8", 2, 32, 1, 64)
    kept = src.evict_into(dst, 32, sink=1, recent=1)
    torch.cuda.synchronize()
    check()
    check_dst()
    assert src.device_status() == tg.TG_STATUS_CACHE_LENGTH
    assert dst.lengths.tolist() == [32, 0] and kept[1].tolist() == [-1] * 32
    assert kept[0].tolist() == ref.kept_slots(w[0].tolist(), 64, 32, 1, 1)
    src.reserve()[:4].zero_()                               # the status word
    q = torch.zeros(2, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    out = src.decode(q)
    assert src.device_status() == tg.TG_STATUS_CACHE_LENGTH
    assert bool((out[1] == 0).all()) and bool(torch.isfinite(out.float()).all())
