"""The 8-bit cache's kernels over the whole range of scales and biases, against the 64-bit reference (tests/cache_ref.py).

The bounds are those that tests/test_gpu_cache_q8.py derives; where a test needs another, it says why.
"""
import numpy as np
import pytest
import torch

from learned_token_pruning_tg_b200 import tokengate as tg
from learned_token_pruning_tg_b200.cache import KVCacheQ8
from tests import cache_ref as ref
from tests.test_gpu_cache_q8 import FORMATS, check_decode, guarded_cache, half_step, ints, random_cache, same_numbers

pytestmark = pytest.mark.gpu

# A block of a sequence in one thread block of 12 warps is a warp's every twelfth one, in a cluster of 16 every 192nd; in
# runs a warp's blocks follow one another.  (B, tokens, max_len, blocks that share an entry of a pattern)
LAUNCHES = {"one thread block": (1, 32 * 72 - 5, 1, 12), "cluster": (1, 32 * 768 - 5, 0, 192), "runs": (160, 32 * 40 - 5, 0, 1)}
ZERO = None                              # a block of zeros, under the least scale, as an append leaves it


def scaled_values(cache, nums, exponents, lens, fmt):
    """V's blocks under 2^exponents[j] (ZERO: zeros under 2^-126) instead of their own scales."""
    B, cap, H, d = cache.v.shape
    codes, scale = cache.v.clone(), torch.full((B, cap // 32, H), float("nan"))
    for j, e in enumerate(exponents):
        if e is ZERO:
            codes[:, 32 * j: 32 * j + 32] = 0
        scale[:, j] = 2.0 ** (-126 if e is ZERO else e)
    for b in range(B):
        codes.view(torch.uint8)[b, lens[b]:] = 0x7f
    cache.v.copy_(codes)
    cache.v_scale.copy_(scale)
    nums["v"] = ref.values(np.nan_to_num(ref.code_values(codes)), np.nan_to_num(scale.double().numpy()))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("pattern", [
    (-6, ZERO, ZERO, -6, ZERO, -6), (-6, -6, ZERO, ZERO, ZERO, ZERO), (ZERO, ZERO, -6, ZERO, ZERO, ZERO),
    (0, -40, -80, -100, -20, 3), (-100, -60, -20, 20, 60, 90), (60, -60, 60, -60, 0, -60), (0, -4, -8, -12, -16, -40),
], ids=str)
@pytest.mark.parametrize("launch", LAUNCHES)
def test_decode_values_of_far_scales(fmt, pattern, launch):
    """Blocks of V whose scales lie far apart, and blocks of zeros, one after the other in a warp."""
    B, T, max_len, every = LAUNCHES[launch]
    lens = [T - 32 * (b % 3) for b in range(B)]
    cache, check, nums, s, w, g = random_cache(fmt, B, T + 5, 1, 64, lens, seed=len(launch))
    scaled_values(cache, nums, [pattern[j // every % 6] for j in range((T + 5) // 32)], lens, fmt)
    q = torch.randn(B, 1, 3, 64, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, 2 * torch.rand(3, generator=g), 1.2, lens, max_len=max_len)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("launch", LAUNCHES)
def test_decode_small_values_behind_masked_large_ones(fmt, launch):
    """The blocks of the largest scale are masked by a bias of -inf: the answer is the small ones'."""
    B, T, max_len, every = LAUNCHES[launch]
    lens = [T] * B
    cache, check, nums, s, w, g = random_cache(fmt, B, T + 5, 2, 64, lens, seed=3)
    exponents = [(0, -100, -90)[j // every % 3] for j in range((T + 5) // 32)]
    scaled_values(cache, nums, exponents, lens, fmt)
    mask = torch.tensor([e == 0 for e in exponents]).repeat_interleave(32)[:T]
    s[:, :T] = torch.where(mask, float("-inf"), s[:, :T])
    cache.s.copy_(s)
    q = torch.randn(B, 1, 4, 64, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, torch.full((4,), 1.25), 1.2, lens, max_len=max_len)


def test_decode_over_appended_zeros():
    """A prompt whose middle is padding of zero rows, as the append itself lays it out, without and with the padding masked."""
    B, T, H, d = 1, 200000, 2, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    cache = KVCacheQ8(B, T, H, d)
    cache.lengths.fill_(T)
    x = torch.randn(2, B, T, H, d, generator=g, device="cuda").to(torch.bfloat16)
    x[:, :, 3000:3400] = 0
    x[1, :, 20000:20100, 1] = 0
    q = torch.randn(B, 1, 4, d, generator=g, device="cuda").to(torch.bfloat16)
    gain = torch.ones(4, device="cuda")
    s = torch.zeros(B, T, device="cuda")
    for masked in (False, True):
        if masked:
            s[:, 3000:3400] = float("-inf")
        cache.append(x[0], x[1], s=s)
        out = cache.decode(q, gain=gain)
        assert cache.device_status() == 0
        k, v = (ref.values(ref.code_values(c), sc.double().cpu().numpy()) for c, sc in
                ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        want, _, _, mass, size = ref.decode(k, v, [T], q.double().cpu().numpy(), s.double().cpu().numpy(), np.ones(4), 1.0)
        e = (d + 8) * 2.0 ** -23 * size
        err = np.abs(out.double().cpu().numpy() - want)
        bound = (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(want) + 2.0 ** -10 * mass)
        assert np.all(err <= bound)


# ------------------------------------------------------------------------------------------- scales of V near fp32's ends
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("e", [100, 110, 117])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_decode_large_values(fmt, e, launch):
    """Values near the largest that an append stores: the answer is finite, whatever the keys' number."""
    B, T, max_len, every = LAUNCHES[launch]
    lens = [T] * B
    cache, check, nums, s, w, g = random_cache(fmt, B, T + 5, 1, 64, lens, seed=4)
    scaled_values(cache, nums, [e - j % 3 for j in range((T + 5) // 32)], lens, fmt)
    q = torch.randn(B, 1, 3, 64, generator=g).to(torch.bfloat16)
    check_decode(cache, check, nums, s, w, q, 2 * torch.rand(3, generator=g), 1.2, lens, max_len=max_len)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [1.5 * 2.0 ** 126, 2.0 ** 127, 1.75 * 2.0 ** 127, 1.25 * 2.0 ** -126, 2.0 ** -130, 2.0 ** -140])
def test_decode_scales_at_the_ends(fmt, scale):
    """Any positive finite scale of V, fp32's largest and its subnormals among them (codes such that the values are finite).
    An answer among bf16's subnormals is half a step of 2^-133 off at most, and the sums' fp32 below 2^-126 a
    few steps of 2^-149: 2^-133 covers both."""
    lens = [900]
    cache, check, nums, s, w, g = random_cache(fmt, 1, 928, 1, 64, lens, seed=6)
    codes = torch.sign(torch.randn(1, 928, 1, 64, generator=g)) * (1.0 if scale > 1 else 96.0)
    if scale > 1:
        codes[:, :, :, ::2] = 0
    cache.v.copy_(codes.to(ref.DTYPE[fmt]))
    cache.v_scale.fill_(scale)
    v = codes.double().numpy() * float(torch.tensor(scale, dtype=torch.float32))
    q = torch.randn(1, 1, 3, 64, generator=g).to(torch.bfloat16)
    gain = torch.rand(3, generator=g)
    out = cache.decode(q.cuda(), gain=gain.cuda(), tau=1.1).double().cpu().numpy()
    want, _, _, mass, size = ref.decode(nums["k"], v, lens, q.double().numpy(), s.double().numpy(), gain.double().numpy(), 1.1)
    e = (64 + 8) * 2.0 ** -23 * size
    bound = (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(want) + 2.0 ** -10 * mass) + 2.0 ** -133
    assert np.all(np.abs(out - want) <= bound)


# ------------------------------------------------------------------------------------------- eviction of zeros
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [1.0, 2.0 ** 12, 2.0 ** 100])
def test_evict_rows_of_zeros(fmt, size):
    """Rows of zeros that leave a block of large numbers: zeros, under the least scale where a new block has no others."""
    B, T, H, d, budget = 1, 128, 2, 64, 40
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(2, B, T, H, d, generator=g) * size).to(torch.bfloat16)
    keep = torch.arange(1, 2 * budget, 2)
    x[:, :, keep] = 0
    x[0, 0, keep[35], 1, 3] = 2.0 ** -100                      # one of the second new block's K rows is not quite zero
    src, dst = KVCacheQ8(B, T, H, d, fmt=fmt), guarded_cache(fmt, B, 64, H, d)[0]
    src.lengths.fill_(T)
    src.append(x[0].cuda(), x[1].cuda())
    src.w[0, keep] = 1.0
    nums = [ref.values(ref.code_values(c), sc.double().cpu().numpy()) for c, sc in ((src.k, src.k_scale), (src.v, src.v_scale))]
    kept = src.evict_into(dst, budget)
    assert kept[0].tolist() == keep.tolist()
    for num, codes, scale in zip(nums, (dst.k, dst.v), (dst.k_scale, dst.v_scale)):
        want, want_scale = ref.append(np.zeros((1, 64, H, d)), np.zeros((1, 2, H)), [budget], [budget], num[:, keep], fmt)
        same_numbers(codes[:, :budget], want[:, :budget])
        assert np.array_equal(scale.double().cpu().numpy(), want_scale)


# ------------------------------------------------------------------------------------------- NaN of a token not seen
@pytest.mark.parametrize("launch", LAUNCHES)
@pytest.mark.parametrize("cut", [5, 30, 3, 0])
@pytest.mark.parametrize("n_q", [2, 4, 16])
def test_decode_nan_value_of_an_unseen_token(launch, cut, n_q):
    """A NaN in V of one of the last tokens gives NaN in its own place of the queries that see the token, and in no other."""
    B, T, max_len, _ = LAUNCHES[launch]
    T = T + 5 - cut
    lens = [T] * B
    cache, check, nums, s, w, g = random_cache("e4m3", B, T + cut, 1, 64, lens, seed=n_q + cut)
    places = [(T - 1, 9), (T - max(n_q // 2, 1), 40)]
    for c, x in places:
        cache.v.view(torch.uint8)[:, c, 0, x] = 0xff if x == 40 else 0x7f
        nums["v"][:, c, 0, x] = np.nan
    q = torch.randn(B, n_q, 1, 64, generator=g).to(torch.bfloat16)
    gain = torch.ones(1)
    lse = torch.empty(B, n_q, 1, device="cuda")
    out = cache.decode(q.cuda(), gain=gain.cuda(), tau=1.2, lse=lse, max_len=max_len).double().cpu().numpy()
    want, want_lse, _, mass, size = ref.decode(nums["k"], nums["v"], lens, q.double().numpy(), s.double().numpy(),
                                               gain.double().numpy(), 1.2)
    nan = np.isnan(want)
    assert nan[:, -1, 0, 9].all() and not nan[:, 0].any() and nan.any(axis=(1, 2)).sum() == 2 * B
    assert np.array_equal(np.isnan(out), nan)
    e = (64 + 8) * 2.0 ** -23 * size
    bound = (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(np.nan_to_num(want)) + 2.0 ** -10 * np.nan_to_num(mass))
    assert np.all(np.abs(out - want)[~nan] <= bound[~nan])
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= e + 2.0 ** -20 + 2.0 ** -23 * np.abs(want_lse))


# ------------------------------------------------------------------------------------------- biases of the lowest number
@pytest.mark.parametrize("gain", [1.0, 0.9, 0.5])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_decode_rows_of_the_lowest_bias(launch, gain):
    """Every key biased by fp32's lowest number (a common mask): the logits are finite and equal, so all keys share the
    weight.  q.k vanishes beside the bias on both sides, so the logits have no error; the rest of the bounds as derived
    (the sums' fp32 2^-20, a weight 2^-18 of itself)."""
    B, T, max_len, _ = LAUNCHES[launch]
    lens = [T - 32 * (b % 3) for b in range(B)]
    cache, check, nums, s, w, g = random_cache("e4m3", B, T + 5, 1, 64, lens, seed=5)
    low = torch.finfo(torch.float32).min
    for b in range(B):
        s[b, :lens[b]] = low
    cache.s.copy_(s)
    w.zero_()
    cache.w.copy_(w)
    q = torch.randn(B, 1, 2, 64, generator=g).to(torch.bfloat16)
    lse = torch.empty(B, 1, 2, device="cuda")
    out = cache.decode(q.cuda(), gain=torch.full((2,), gain, device="cuda"), lse=lse, accumulate=True, max_len=max_len)
    n = np.array(lens, dtype=np.float64)[:, None]
    v = [nums["v"][b, :lens[b], 0] for b in range(B)]
    want, mass = np.stack([x.mean(0) for x in v])[:, None, None], np.stack([np.abs(x).mean(0) for x in v])[:, None, None]
    bound = (2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(want) + 2.0 ** -10 * mass)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= bound)
    want_lse = float(torch.tensor(gain)) * low
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 2.0 ** -23 * abs(want_lse))
    got = cache.w.double().cpu().numpy()
    for b in range(B):
        assert np.all(np.abs(got[b, :lens[b]] - 2 / n[b]) <= 2.0 ** -18 * 2 / n[b])
    check()


# ------------------------------------------------------------------------------------------- status
def test_status_of_earlier_calls_stays():
    """What an append flagged is still there when a decode has made the workspace larger, and when a graph captured on the
    smaller one runs once more."""
    cache = KVCacheQ8(1, 64, 1, 64)
    x = torch.ones(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    bad = x.clone()
    bad[..., 3] = float("inf")
    cache.lengths.fill_(1)
    cache.append(bad, x)
    q = torch.ones(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache.decode(q)
    assert cache.device_status() == tg.TG_STATUS_CACHE_VALUE
    cache.decode(q, accumulate=True)
    assert cache.device_status() == tg.TG_STATUS_CACHE_VALUE

    cache = KVCacheQ8(1, 64, 1, 64)
    cache.lengths.fill_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append(x, x)
    cache.decode(q)
    assert cache.device_status() == 0
    cache.lengths.fill_(65)
    graph.replay()
    torch.cuda.synchronize()
    assert cache.device_status() == tg.TG_STATUS_CACHE_LENGTH


# ------------------------------------------------------------------------------------------- lengths
def test_read_with_the_lowest_length():
    """A length of int32's lowest number reads nothing, from wherever the read begins."""
    cache, check, nums, s, w, g = random_cache("int8", 2, 320, 2, 64, [300, 300], seed=1)
    cache.lengths.copy_(ints([-2 ** 31, 300]))
    for first in (0, 1, 64):
        out = [torch.full((2, 320 - first, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        cache.read(*out, first=first)
        torch.cuda.synchronize()
        check()
        assert bool((out[0][0] == 7).all()) and bool((out[1][0] == 7).all())
        assert np.array_equal(out[0][1, :300 - first].double().cpu().numpy(), nums["k"][1, first:300])


# ------------------------------------------------------------------------------------------- NaN of a masked token
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("launch", LAUNCHES)
def test_decode_nan_value_of_a_masked_token(launch, rest):
    """A NaN in V of a key that a bias of -inf masks is a NaN in its place (0 times NaN), whichever keys share its warp:
    among masked keys all around it, with other keys (rest) or none that count."""
    B, T, max_len, _ = LAUNCHES[launch]
    lens = [T] * B
    cache, check, nums, s, w, g = random_cache("e4m3", B, T + 5, 1, 64, lens, seed=9)
    s[:, T // 4: T] = float("-inf")
    if not rest:
        s[:, :T] = float("-inf")
    cache.s.copy_(s)
    at = T // 2 + 3
    cache.v.view(torch.uint8)[:, at, 0, 21] = 0x7f
    q = torch.randn(B, 1, 3, 64, generator=g).to(torch.bfloat16)
    out = cache.decode(q.cuda(), gain=torch.full((3,), 0.8, device="cuda"), tau=1.2, max_len=max_len).double().cpu().numpy()
    nan = np.zeros(out.shape, dtype=bool)
    nan[..., 21] = True
    assert np.array_equal(np.isnan(out), nan)
    want, _, _, mass, size = ref.decode(nums["k"], nums["v"], lens, q.double().numpy(), s.double().numpy(), np.full(3, np.float32(0.8)), 1.2)
    e = (64 + 8) * 2.0 ** -23 * size
    bound = (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(want) + 2.0 ** -10 * mass)
    assert np.all(np.abs(out - want)[~nan] <= bound[~nan])
    assert rest or not out[~nan].any()
