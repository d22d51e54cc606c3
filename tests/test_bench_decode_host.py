"""Host-side pieces of the decode benches (no GPU)."""
import bench


def test_caches_in_turn_are_twice_the_l2():
    bf16 = 2 * 65537 * 8 * 128 * 2 + 65537 * 4
    eight = 2 * 65537 * 8 * 128 + 2 * 2049 * 8 * 4 + 65537 * 4
    assert bench.caches_in_turn(bf16) == 1 and bench.caches_in_turn(eight) == 2
    for nbytes in (1 << 20, eight, bf16, 2 * bench.L2_BYTES, 1 << 30):
        n = bench.caches_in_turn(nbytes)
        assert n * nbytes >= 2 * bench.L2_BYTES and (n == 1 or (n - 1) * nbytes < 2 * bench.L2_BYTES)
