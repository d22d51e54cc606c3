"""The 8-bit cache without a GPU: the tests' own formats against torch, and every refusal of its calls (C and Python)."""
import ctypes

import numpy as np
import pytest
import torch

from learned_token_pruning_tg_b200 import build as tg_build
from learned_token_pruning_tg_b200 import cache as tgc
from learned_token_pruning_tg_b200 import tokengate as tg
from tests import cache_ref as ref

INV, UNS, OK = tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED, tg.TG_OK


@pytest.fixture(scope="module")
def lib():
    tg_build.build()
    return tg.lib()


def test_reference_e4m3_is_the_format():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn)
    want = codes.float().double().numpy()
    got = ref.e4m3_values()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_reference_rounding():
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(4000, generator=g) * 100, torch.randn(4000, generator=g) * 0.01,
                   torch.tensor([0.0, 17.0, 18.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, -448.0])]).clamp(-448, 448)
    assert np.array_equal(ref.to_code_value(x.numpy(), "e4m3"), x.to(torch.float8_e4m3fn).float().double().numpy())
    y = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.0])
    assert ref.to_code_value(y.numpy(), "int8").tolist() == [0.0, 2.0, 2.0, -0.0, -2.0, 126.0, 127.0]


def test_reference_scale():
    assert ref.scale_of(448.0, "e4m3") == 1.0 and ref.scale_of(449.0, "e4m3") == 2.0
    assert ref.scale_of(224.0, "e4m3") == 0.5 and ref.scale_of(0.0, "e4m3") == 2.0 ** -126
    assert ref.scale_of(127.0, "int8") == 1.0 and ref.scale_of(127.5, "int8") == 2.0


def test_reference_kept_slots():
    nan = float("nan")
    assert ref.kept_slots([0, 5, 1, 5, nan, 2, 9], 7, 4, 1, 1) == [0, 1, 3, 6]
    assert ref.kept_slots([0, nan, -1, 0], 4, 2, 0, 0) == [0, 3]
    assert ref.kept_slots([1, 2], 2, 5, 1, 1) == [0, 1]


def test_growing_a_scale_by_parts():
    # token by token: each growth rounds the earlier codes once more; never off by more than the last scale's step
    x = torch.tensor([[[[1.0]], [[100.0]], [[3.0]], [[2000.0]]]]).expand(1, 4, 1, 64).numpy()
    codes, scale = np.zeros((1, 32, 1, 64)), np.zeros((1, 1, 1))
    for i in range(4):
        codes, scale = ref.append(codes, scale, [i + 1], [1], x[:, i: i + 1], "int8")
    assert scale[0, 0, 0] == 16.0 and codes[0, :4, 0, 0].tolist() == [0.0, 6.0, 0.0, 125.0]


def struct(**kw):
    d = dict(format=0, batch=2, Hkv=2, d_h=128, capacity=64, ld_token=256, ld_seq=64 * 256, k=4096, v=1 << 20,
             k_scale=1 << 21, v_scale=1 << 22, lengths=1 << 23, s=None, w=1 << 24)
    d.update(kw)
    return tg.CacheStruct(**d)


def test_cache_struct_refusals(lib):
    def read(**kw):
        c = struct(**kw)
        return lib.tg_cache_read_q8(ctypes.byref(c), 0, 0, None, None, None)   # n = 0: nothing is launched

    assert read() == OK
    assert read(batch=0, k=None, v=None, k_scale=None, v_scale=None, lengths=None) == OK
    assert lib.tg_cache_read_q8(None, 0, 0, None, None, None) == INV
    for bad in (dict(format=2), dict(format=-1), dict(batch=-1), dict(capacity=-32), dict(capacity=65), dict(Hkv=0),
                dict(ld_token=255), dict(ld_token=128), dict(ld_token=264), dict(ld_seq=63 * 256), dict(ld_seq=64 * 256 + 8),
                dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(lengths=None), dict(k=4100),
                dict(v=8)):
        assert read(**bad) == INV, bad
    for bad in (dict(d_h=96), dict(Hkv=65, ld_token=65 * 128, ld_seq=64 * 65 * 128), dict(batch=65536),
                dict(capacity=1 << 31, ld_seq=1 << 40)):
        assert read(**bad) == UNS, bad
    vp = ctypes.c_void_p
    c = struct()
    r = lambda first, n, k=16, v=16: lib.tg_cache_read_q8(ctypes.byref(c), first, n, vp(k), vp(v), None)  # noqa: E731
    assert r(-1, 1) == INV and r(0, -1) == INV and r(0, 65) == INV and r(64, 1) == INV and r(1 << 62, 1 << 62) == INV
    assert r(0, 1, k=24) == INV and r(0, 1, v=0) == INV


def test_workspace_bytes(lib):
    n = lambda n_q, Hq, acc, **kw: lib.tg_cache_workspace_bytes(ctypes.byref(struct(**kw)), n_q, Hq, acc)  # noqa: E731
    assert n(0, 0, 0) == 256
    small, with_w = n(1, 4, 0), n(1, 4, 1)
    assert 256 < small < with_w and with_w - small == 2 * 2 * 64 * 2 * 4
    assert n(1, 3, 0) == 0                          # Hq % Hkv
    assert n(1, 34, 0) == 0 and n(9, 4, 0) == 0     # more than 16 rows a KV head
    assert n(8, 4, 0) > 0
    assert n(-1, 4, 0) == 0 and n(1, 4, 0, d_h=96) == 0
    assert lib.tg_cache_workspace_bytes(None, 1, 4, 0) == 0
    assert n(1, 4, 1, k=None, lengths=None) == with_w   # sizes alone count


def test_append_refusals(lib):
    vp = ctypes.c_void_p

    def app(c=None, k=16, ld_k=256, ldb_k=1024, v=16, ld_v=256, ldb_v=1024, n=4, ws=256, ws_bytes=256):
        c = c or struct()
        return lib.tg_cache_append_q8(ctypes.byref(c), vp(k), ld_k, ldb_k, vp(v), ld_v, ldb_v, n, None, None, vp(ws),
                                      ws_bytes, None)

    assert app(n=0) == OK and app(c=struct(batch=0)) == OK
    assert app(n=-1) == INV
    assert app(n=1 << 31) == UNS
    assert app(k=0) == INV and app(v=24) == INV and app(ws=0) == INV and app(ws_bytes=255) == INV and app(ws=264) == INV
    assert app(ld_k=252) == INV and app(ld_v=248) == INV and app(ldb_k=1020) == INV and app(ldb_v=128) == INV
    assert app(c=struct(d_h=96)) == UNS


def test_decode_refusals(lib):
    vp = ctypes.c_void_p

    def dec(c=None, q=16, n_q=1, Hq=4, tau=1.0, acc=0, max_len=0, out=1 << 16, ws=256, ws_bytes=1 << 30):
        c = c or struct()
        return lib.tg_gated_decode_q8(ctypes.byref(c), vp(q), n_q, Hq, None, tau, acc, max_len, vp(out), None, vp(ws),
                                      ws_bytes, None)

    assert dec(c=struct(batch=0)) == OK
    assert dec(n_q=0) == INV and dec(Hq=0) == INV and dec(Hq=5) == INV and dec(max_len=-1) == INV
    assert dec(tau=float("nan")) == INV and dec(tau=float("inf")) == INV
    assert dec(Hq=34) == UNS and dec(n_q=9) == UNS and dec(n_q=1 << 30) == UNS
    assert dec(q=4096, out=4096) == INV and dec(q=4096, out=4096 + 1024) == INV    # the answer over the queries
    assert dec(q=0) == INV and dec(q=24) == INV and dec(out=8) == INV and dec(ws=0) == INV
    need = lib.tg_cache_workspace_bytes(ctypes.byref(struct()), 1, 4, 1)
    assert dec(acc=1, ws_bytes=need - 1) == INV
    assert dec(c=struct(w=None), acc=1) == INV


def test_evict_refusals(lib):
    vp = ctypes.c_void_p

    def ev(src=None, dst=None, budget=32, sink=1, recent=4, max_len=0, kept=16, ws=256, ws_bytes=256):
        src = src or struct()
        dst = dst or struct(k=1 << 30, v=1 << 31, k_scale=1 << 32, v_scale=1 << 33, lengths=1 << 34, w=1 << 35)
        return lib.tg_cache_evict_q8(ctypes.byref(src), ctypes.byref(dst), budget, sink, recent, max_len, vp(kept),
                                     vp(ws), ws_bytes, None)

    other = dict(k=1 << 30, v=1 << 31, k_scale=1 << 32, v_scale=1 << 33, lengths=1 << 34, w=1 << 35)
    assert ev(src=struct(batch=0), dst=struct(batch=0, **other)) == OK
    assert ev(budget=-1) == INV and ev(sink=-1) == INV and ev(recent=-1) == INV and ev(max_len=-1) == INV
    assert ev(sink=20, recent=13) == INV                  # more protected tokens than the budget
    assert ev(sink=1 << 62, recent=1 << 62, budget=40) == INV
    assert ev(budget=65) == INV                           # dst is too small
    assert ev(kept=0) == INV and ev(ws=0) == INV and ev(ws_bytes=8) == INV
    assert ev(src=struct(w=None)) == INV
    for bad in (dict(format=1), dict(batch=1), dict(Hkv=1), dict(d_h=64)):
        assert ev(dst=struct(**{**other, **bad})) == INV, bad
    # shared memory between the two caches
    for bad in (dict(k=4096), dict(k=4096 + 64 * 256), dict(v=4096), dict(k=1 << 20), dict(w=(1 << 24) + 256),
                dict(k_scale=1 << 21), dict(v_scale=1 << 22), dict(lengths=1 << 23)):
        assert ev(dst=struct(**{**other, **bad})) == INV, bad


def test_python_refusals():
    z = torch.zeros
    with pytest.raises(TypeError):
        tg.CacheQ8(z(1, 32, 1, 64), z(1, 32, 1, 64), None, None, None)       # not 8-bit codes
    codes = z(1, 32, 1, 64, dtype=torch.int8)
    with pytest.raises(TypeError, match="CUDA"):
        tg.CacheQ8(codes, codes, z(1, 1, 1), z(1, 1, 1), z(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="fmt"):
        tgc.KVCacheQ8(1, 32, 1, 64, fmt="e5m2")
