"""Work sharing of the weight gradient from 8 bits, checked on the host through the
library's own schedule code (no GPU needed): every slice of every tile is summed
exactly once, a split tile is held by consecutive pairs in row order, no pair uses
a partial-sum slot twice, and the shares are even."""
import collections

import pytest

from dense_gemm_07_gb300 import _abi

# (T, K, N, resident pairs)
CASES = [
    (4096, 4096, 11008, 76),  # 688 tiles: 9 whole waves and 4 tiles
    (4096, 128, 256, 76),     # one tile over two pairs
    (8321, 1000, 3001, 76),   # 48 tiles over 76 pairs: two and three segments
    (8320, 1000, 3001, 76),   # the same tiles, a slice short of a split
    (3001, 1000, 3001, 76),
    (4096, 2816, 2048, 76),   # 88 tiles, all of them shared
    (3500, 4096, 2560, 76),   # one whole wave, 84 tiles shared
    (4096, 256 * 76, 256, 76),   # a whole wave
    (130, 2560, 2100, 76),    # two slices: never split
    (100000, 300, 200, 76),   # two tiles, a long sum
    (9999, 513, 1025, 7),     # other resident counts
    (9999, 513, 1025, 1),
    (1, 1, 1, 76),
]


def _tiles(K, N):
    return (K + 255) // 256 * ((N + 255) // 256)


def _units(T, K, N, P):
    return {p: _abi.gemm_ckpt8_wgrad_units(T, K, N, P, p) for p in range(P)}


@pytest.mark.parametrize("T,K,N,P", CASES)
def test_every_slice_exactly_once(T, K, N, P):
    slices = (T + 127) // 128
    cover = collections.defaultdict(list)
    for p, units in _units(T, K, N, P).items():
        for tile, k0, k1, slot, first, nseg, shared, n_off, width in units:
            assert 0 <= k0 < k1 <= slices and (n_off, width) == (0, 256)
            cover[tile].append((k0, k1, p, slot, first, nseg, shared))
    assert sorted(cover) == list(range(_tiles(K, N)))
    for tile, segs in cover.items():
        segs.sort()
        assert segs[0][0] == 0 and segs[-1][1] == slices
        assert all(a[1] == b[0] for a, b in zip(segs, segs[1:]))
        if len(segs) == 1:
            assert segs[0][3:6] == (-1, segs[0][2], 1)
            continue
        pairs = [s[2] for s in segs]
        assert pairs == list(range(pairs[0], pairs[0] + len(pairs))) and len(segs) <= 3
        assert all(s[4] == pairs[0] and s[5] == len(segs) and s[6] == 1 for s in segs)


@pytest.mark.parametrize("T,K,N,P", CASES)
def test_slots_and_shares(T, K, N, P):
    slices = (T + 127) // 128
    shares = []
    for units in _units(T, K, N, P).values():
        slots = [u[3] for u in units if u[3] >= 0]
        assert len(set(slots)) == len(slots) and set(slots) <= {0, 1}
        flags = [u[6] for u in units]
        assert flags == sorted(flags)  # whole tiles come first
        shared = sum(u[2] - u[1] for u in units if u[6])
        if shared:
            shares.append(shared)
    if shares:
        assert max(shares) - min(shares) <= 1
        assert min(shares) >= slices // 2  # so a tile has at most three segments


def test_what_is_split():
    def split(T, K, N):
        units = _units(T, K, N, 76)
        return (sum(u[6] == 0 for us in units.values() for u in us),
                len({u[0] for us in units.values() for u in us if u[6]}),
                {u[5] for us in units.values() for u in us if u[6]})
    assert split(4096, 128, 256) == (0, 1, {2})
    assert split(8321, 1000, 3001) == (0, 48, {2, 3})
    assert split(8320, 1000, 3001) == (48, 0, set())
    assert split(4096, 2816, 2048) == (0, 88, {1, 2})
    assert split(3500, 4096, 2560) == (76, 84, {1, 2})
    assert split(130, 2560, 2100) == (90, 0, set())


def test_bad_arguments():
    for args in [(0, 4, 4, 76, 0), (4, -1, 4, 76, 0), (4, 4, 0, 76, 0), (4, 4, 4, 0, 0),
                 (4, 4, 4, 76, 76), (4, 4, 4, 76, -1), (4, 2 ** 31 - 1, 2 ** 31 - 1, 76, 0)]:
        with pytest.raises(ValueError):
            _abi.gemm_ckpt8_wgrad_units(*args)
