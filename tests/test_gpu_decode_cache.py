"""The 8-bit cache's operators as a decoding program runs them together, behind a pruned prefill.

The stack's prefill leaves keys, values and the kept tokens' scores; its caches are taken over in 8 bits, and some steps
run on them: the new token's key and value appended, attention with the weights gathered, and, when the caches are
full, the lightest tokens evicted into other caches, on which decoding goes on.  Everything is checked step by step against the
64-bit reference fed with the same rows; the attention within the bound of its inputs' own 8 bits is the formula's
(tests/test_gpu_cache_q8.py derives it).
"""
import numpy as np
import pytest
import torch

from learned_token_pruning_tg_b200 import stack as stk
from learned_token_pruning_tg_b200.cache import KVCacheQ8
from tests import cache_ref as ref
from tests.test_gpu_cache_q8 import half_step, same_numbers

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_decode_behind_a_pruned_prefill(fmt):
    cfg = stk.STACK_TINY
    wts = stk.random_weights(cfg, "cuda")
    s = stk.PrunedPrefillStack(cfg, wts)
    s.run(stk.random_embeddings(cfg, "cuda"), prune=True, keep_kv=True)
    extra = 40
    caches = s.decode_caches(extra, fmt=fmt)
    assert len(caches) == cfg.n_layers
    assert caches[0].lengths is caches[1].lengths and caches[2].lengths is caches[3].lengths
    assert [int(c.lengths) for c in caches] == [cfg.N, cfg.N, cfg.K, cfg.K]
    for (k, v, sc), c in zip(s.kv, caches):
        n = k.shape[0]
        for x, codes, scale in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
            cap = codes.shape[1]
            want, want_scale = ref.append(np.zeros((1, cap, cfg.Hkv, cfg.d_h)), np.zeros((1, cap // 32, cfg.Hkv)), [n], [n],
                                          x[None].double().cpu().numpy(), fmt)
            same_numbers(codes, want)
            assert np.array_equal(scale.double().cpu().numpy()[:, : -(-n // 32)], want_scale[:, : -(-n // 32)])
        assert torch.equal(c.s[0, :n], torch.zeros_like(c.s[0, :n]) if sc is None else sc)

    # decode on one layer above the gate
    li = cfg.gate_layer + 1
    cache, gain, tau = caches[li], wts.layers[li].gain, wts.layers[li].tau
    other = KVCacheQ8(1, cfg.K + extra, cfg.Hkv, cfg.d_h, fmt=fmt, lengths=torch.zeros_like(cache.lengths))
    g = torch.Generator().manual_seed(1)
    state = {m: (ref.code_values(t), sc.double().cpu().numpy())
             for m, t, sc in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale))}
    sb, wb, n = cache.s[0].double().cpu().numpy(), np.zeros(cache.capacity), cfg.K
    for step in range(60):
        q, k, v = (torch.randn(1, 1, h, cfg.d_h, generator=g).to(torch.bfloat16)
                   for h in (cfg.Hq, cfg.Hkv, cfg.Hkv))
        sc = torch.randn(1, 1, generator=g)
        n += 1
        cache.lengths.add_(1)
        cache.append(k.cuda(), v.cuda(), s=sc.cuda())
        lse = torch.empty(1, 1, cfg.Hq, device="cuda")
        out = cache.decode(q.cuda(), gain=gain, tau=tau, lse=lse, accumulate=True)
        for m, x in (("k", k), ("v", v)):
            state[m] = ref.append(*state[m], [n], [1], x.double().numpy(), fmt)
        sb[n - 1], wb[n - 1] = float(sc), 0.0
        kk, vv = (ref.values(*state[m]) for m in ("k", "v"))
        want, want_lse, want_w, mass, size = ref.decode(kk, vv, [n], q.double().numpy(), sb[None],
                                                        gain.double().cpu().numpy(), tau)
        wb += want_w[0]
        e = (cfg.d_h + 8) * 2.0 ** -23 * size
        err = np.abs(out.double().cpu().numpy() - want)
        bound = (2 * e + 2.0 ** -12 + 2.0 ** -19) * mass * (1 + 2.0 ** -8) + half_step(np.abs(want) + 2.0 ** -10 * mass)
        assert np.all(err <= bound), (step, np.max(err - bound))
        assert np.max(np.abs(lse.double().cpu().numpy() - want_lse)) <= e + 2.0 ** -20 + 2.0 ** -23 * np.max(np.abs(want_lse))
        # weights of 60 steps' rounding at most
        got_w = cache.w[0].double().cpu().numpy()
        assert np.all(np.abs(got_w[:n] - wb[:n]) <= 60 * (2 * e + 2.0 ** -18) * wb[:n] + 1e-30)
        if n == cfg.K + extra:                              # full: the heaviest half and the last 32 stay
            budget, sink, recent = cfg.K // 2, 4, 32
            kept = cache.evict_into(other, budget, sink=sink, recent=recent)
            slots = ref.kept_slots(got_w[:n].tolist(), n, budget, sink, recent)
            assert kept[0].tolist() == slots and int(other.lengths) == budget
            for m, t in (("k", other.k), ("v", other.v)):
                num = ref.values(*state[m])
                state[m] = ref.append(np.zeros(t.shape), np.zeros((1, t.shape[1] // 32, cfg.Hkv)), [budget], [budget],
                                      num[:, slots], fmt)
                same_numbers(t, state[m][0])
            sb = np.concatenate([sb[slots], np.zeros(other.capacity - budget)])
            wb = np.concatenate([got_w[slots], np.zeros(other.capacity - budget)])
            cache, other, n = other, cache, budget
    assert cache.device_status() == 0 and other.device_status() == 0


@pytest.mark.parametrize("fmt,tol", [("e4m3", 2.0 ** -4), ("int8", 0.5 / 63)])
def test_reads_back_what_the_other_cache_takes(fmt, tol):
    """The values read back decode in tg_gated_decode as the codes do here, and lie within the format's step of what was
    appended: e4m3 half a step of its own number (2^-4) or of the least exponent's (2^-10 of the scale, below 2^-17 of
    the block's largest), int8 half a step of at most 1/63 of the block's largest number."""
    from learned_token_pruning_tg_b200 import tokengate as tg
    T, H, Hq, d = 1000, 2, 4, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(1, T, H, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    s = torch.randn(1, T, generator=g, device="cuda")
    cache = KVCacheQ8(1, T, H, d, fmt=fmt)
    cache.lengths.fill_(T)
    cache.append(k, v, s=s)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    cache.read(ko, vo)
    for x, y in ((k, ko), (v, vo)):
        pad = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, -T % 32)).view(1, -1, 32, H, d)
        top = pad.abs().amax((2, 4)).repeat_interleave(32, 1)[:, :T, :, None]
        err = (x.float() - y.float()).abs()
        size = x.float().abs() if fmt == "e4m3" else top
        assert bool((err <= tol * size + 2.0 ** -17 * top).all())
    q = torch.randn(1, 1, Hq, d, generator=g, device="cuda").to(torch.bfloat16)
    gain = torch.rand(Hq, generator=g, device="cuda")
    out = cache.decode(q, gain=gain, tau=1.1)
    want = torch.empty(Hq, d, dtype=torch.bfloat16, device="cuda")
    tg.tg_gated_decode(q[0, 0], ko[0], vo[0], want, tg.new_workspace(0, Hq, op=tg.TG_OP_DECODE), s_cache=s[0], gain=gain, tau=1.1)
    # the same cache in both: P's fp16 here (2^-12 of sum p |v| <= 2^-12 max |v|) and a rounding to bf16 each
    diff = (out[0, 0].float() - want.float()).abs()
    assert bool((diff <= 2.0 ** -8 * want.float().abs() + 2.0 ** -11 * vo.float().abs().max()).all())
