"""CPU tests of the segment length that kda_linear_seg_len chooses: every length covers its axis, and no other equal
cut has a much shorter critical path."""
import ctypes
import math

import pytest

from gated_delta_rule_pack_amd import _lib


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _sizes(T, H, N=1, K=128, V=128, es=4):
    """Sizes alone: nothing is read, and the addresses are far apart."""
    a = _lib.LinearArgs()
    a.T, a.N, a.H, a.H_qk, a.K, a.V, a.scale = T, N, H, H, K, V, 1.0
    a.q, a.k, a.v, a.out, a.cu_seqlens = (i << 42 for i in range(1, 6))
    a.state_cache, a.num_slots, a.state_cache_stride0 = 6 << 42, N, H * K * V
    a.state_indices, a.has_initial_state = 7 << 42, 8 << 42
    a.state_dtype = _lib.KDA_F32 if es == 4 else _lib.KDA_BF16
    return a, T + (N - 1) * (K * V * es * 2 // ((K + V) * 4))  # a state counts as the tokens whose bytes it costs


SHAPES = [(T, H) for T in (1024, 4096, 16384, 53000, 65536) for H in (1, 2, 3, 7, 12, 20, 32, 40, 48, 64, 96, 100, 128, 160, 192,
                                                                      224, 255, 256, 300, 512)]
# Those whose segments make more workgroups than the 256 compute units, before the length is settled.
CROWDED = [(T, H) for T, H in SHAPES if H >= 20] + [(53000, 2), (65536, 2), (65536, 3)]


def _path(axis, n, H, plane):
    """Tokens' walks that the fullest of 256 compute units makes, one after the other, in the time of an output walk
    of 64 (3 us; 2 more where there is a map walk), and the combine's chain: a segment costs it 0.06 us, and each
    head's state 0.059."""
    work = -(-n * H // 256) * -(-axis // n) / 64
    return work * 3 if n == 1 else work * 5 + n * (0.06 + 0.059 * H * plane)


@pytest.mark.parametrize("T,H", CROWDED)
def test_no_other_cut_is_much_shorter(lib, T, H):
    """At V = 128, where two workgroups share a compute unit: within 1.4 (chunks are whole, and the model counts a
    compute unit with two as twice as slow, where it is up to a third faster)."""
    a, axis = _sizes(T, H)
    L = lib.kda_linear_seg_len(ctypes.byref(a))
    n = -(-axis // L)
    best = min(range(1, max(1, 512 // H) + 1), key=lambda m: _path(axis, m, H, 1.0))
    got, least = _path(n * L, n, H, 1.0), _path(axis, best, H, 1.0)
    print(f"  T={T} H={H}: {n} segments of {L}, {got:.0f}; best {best}, {least:.0f}")
    assert got <= 1.4 * least


@pytest.mark.parametrize("K,V,es", [(128, 128, 4), (128, 64, 4), (64, 64, 2)])
@pytest.mark.parametrize("N", [1, 5, 128])
@pytest.mark.parametrize("T,H", SHAPES[::3])
def test_segments_cover_the_axis(lib, T, H, N, K, V, es):
    a, axis = _sizes(T, H, N, K, V, es)
    L = lib.kda_linear_seg_len(ctypes.byref(a))
    n = -(-axis // L)
    assert L > 0 and L % 64 == 0 and (n - 1) * L < axis <= n * L
