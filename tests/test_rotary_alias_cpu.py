"""CPU tests of which memory kda_rotary accepts: results in place or without an element in common with anything else,
byte ranges interleaved or not."""
import ctypes
import random

import pytest
import torch

import gated_delta_rule_pack_amd as kda
from gated_delta_rule_pack_amd import _lib

BASE = 1 << 40  # stands for the buffer; nothing is read
ES = 2


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _status(lib, T, D, Hq, Hk, q, k, oq, ok):
    """q, k, oq, ok: (first element, token stride, head stride)."""
    a = _lib.RotaryArgs()
    a.T, a.D, a.H_q, a.H_k, a.rot_dim, a.dtype, a.factor = T, D, Hq, Hk, 2, _lib.KDA_BF16, 1.0
    a.positions, a.inv_freq = 1 << 50, 1 << 51
    for name, (at, st, sh) in (("q", q), ("k", k), ("out_q", oq), ("out_k", ok)):
        setattr(a, name, BASE + ES * at)
        setattr(a, f"{name}_stride_t", st)
        setattr(a, f"{name}_stride_h", sh)
    return lib.kda_rotary_validate(ctypes.byref(a))


def _elements(T, H, D, rows):
    at, st, sh = rows
    return {at + t * st + h * sh + d for t in range(T) for h in range(H) for d in range(D)}


FAR = 1 << 24  # a buffer of its own
T, D = 20, 64


LAYOUTS = {
    # name: (Hq, Hk, q, k, out_q, out_k), accepted
    "results are columns of one buffer": ((4, 2, (FAR, 256, 64), (2 * FAR, 128, 64), (0, 384, 64), (256, 384, 64)), True),
    "the same, wider": ((4, 2, (FAR, 256, 64), (2 * FAR, 128, 64), (8, 512, 64), (264, 512, 64)), True),
    "q in place, k elsewhere": ((4, 2, (0, 512, 64), (256, 512, 64), (0, 512, 64), (FAR, 128, 64)), True),
    "k in place, q elsewhere": ((4, 2, (0, 512, 64), (256, 512, 64), (FAR, 256, 64), (256, 512, 64)), True),
    "k before q": ((4, 2, (128, 512, 64), (0, 512, 64), (128, 512, 64), (FAR, 128, 64)), True),
    "results beside their inputs": ((2, 2, (0, 512, 64), (128, 512, 64), (256, 512, 64), (384, 512, 64)), True),
    "heads of q, k and v in turn, in place": ((3, 3, (0, 576, 192), (64, 576, 192), (0, 576, 192), (64, 576, 192)), True),
    "the same, results in turn": ((3, 3, (FAR, 192, 64), (2 * FAR, 192, 64), (64, 384, 128), (0, 384, 128)), True),
    "heads outside tokens, one buffer": ((2, 2, (FAR, 64, 20 * 64), (2 * FAR, 64, 20 * 64), (0, 64, 2 * 20 * 64), (20 * 64, 64, 2 * 20 * 64)), True),
    "one head of k between those of q": ((3, 1, (FAR, 192, 64), (2 * FAR, 64, 64), (0, 256, 96), (64, 256, 64)), False),
    "k's first head is q's last": ((4, 2, (FAR, 256, 64), (2 * FAR, 128, 64), (0, 384, 64), (192, 384, 64)), False),
    "k's last head is the next token's first": ((4, 2, (FAR, 256, 64), (2 * FAR, 128, 64), (0, 384, 64), (320, 384, 64)), False),
    "q in place shares a head with k": ((4, 2, (0, 512, 64), (192, 512, 64), (0, 512, 64), (FAR, 128, 64)), False),
    "result over the other input": ((4, 2, (0, 512, 64), (256, 512, 64), (256, 512, 64), (FAR, 128, 64)), False),
    "in turn, off by one": ((3, 3, (FAR, 192, 64), (2 * FAR, 192, 64), (63, 384, 128), (0, 384, 128)), False),
    "shifted by a token": ((2, 2, (0, 128, 64), (FAR, 128, 64), (128, 128, 64), (2 * FAR, 128, 64)), False),
    "token strides differ": ((2, 2, (FAR, 128, 64), (2 * FAR, 128, 64), (0, 512, 64), (256, 256, 64)), False),
}


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_layouts(lib, name):
    (Hq, Hk, q, k, oq, ok), accepted = LAYOUTS[name]
    sets = [_elements(T, h, D, r) for h, r in ((Hq, q), (Hk, k), (Hq, oq), (Hk, ok))]
    others = [(2, 1), (3, 0), (2, 3)] + ([] if q == oq else [(2, 0)]) + ([] if k == ok else [(3, 1)])
    apart = all(not sets[i] & sets[j] for i, j in others)
    assert apart == accepted or name == "token strides differ"  # refused although it may be apart
    assert _status(lib, T, D, Hq, Hk, q, k, oq, ok) == (_lib.KDA_OK if accepted else _lib.KDA_ERR_ALIAS)


@pytest.mark.parametrize("seed", range(8))
def test_random_layouts(lib, seed):
    """Against the sets of elements: nothing that meets is accepted, and with equal token strides all that does not is."""
    r = random.Random(seed)
    seen = {True: 0, False: 0}
    while min(seen.values()) < 150:
        T, D, Hq, Hk = r.randint(1, 5), r.choice([2, 3, 4]), r.randint(1, 4), r.randint(1, 4)
        sh = [r.choice([D, D, D + 1, 2 * D, 3 * D, T * D, 2 * T * D]) for _ in range(2)]
        st = r.choice([D, (Hq - 1) * sh[0] + D, (Hk - 1) * sh[1] + D, Hq * sh[0] + Hk * D, 3 * D * max(Hq, Hk), r.randint(D, 60)])
        st = [st, st if r.random() < 0.8 else r.randint(D, 60)]
        oq, ok = (0, st[0], sh[0]), (r.randint(-70, 70), st[1], sh[1])
        alone = [_status(lib, T, D, h, 0, (FAR, Hq * D * 9, D), (0, 0, 0), o, (0, 0, 0)) for h, o in ((Hq, oq), (Hk, ok))]
        if alone != [_lib.KDA_OK] * 2:  # rows of one result meet
            continue
        apart = not _elements(T, Hq, D, oq) & _elements(T, Hk, D, ok)
        got = _status(lib, T, D, Hq, Hk, (FAR, Hq * D, D), (2 * FAR, Hk * D, D), oq, ok)
        equal = T == 1 or st[0] == st[1]
        assert got in (_lib.KDA_OK, _lib.KDA_ERR_ALIAS)
        assert apart or got != _lib.KDA_OK, (T, D, Hq, Hk, oq, ok)
        assert not (apart and equal) or got == _lib.KDA_OK, (T, D, Hq, Hk, oq, ok)
        seen[apart] += 1


def test_one_token_takes_its_place_whatever_its_token_stride(lib):
    assert _status(lib, 1, D, 4, 2, (0, 512, 64), (256, 512, 64), (0, 256, 64), (256, 128, 64)) == _lib.KDA_OK
    assert _status(lib, 1, D, 4, 2, (0, 512, 64), (192, 512, 64), (0, 256, 64), (192, 128, 64)) == _lib.KDA_ERR_ALIAS


def test_binding_passes_columns_of_one_buffer(lib):
    q, k = torch.zeros(20, 4, 64, dtype=torch.bfloat16), torch.zeros(20, 2, 64, dtype=torch.bfloat16)
    both = torch.zeros(20, 6, 64, dtype=torch.bfloat16)
    a = kda.make_rotary_args(q, k, torch.arange(20), torch.ones(8, dtype=torch.float64), both[:, :4], both[:, 4:])
    assert lib.kda_rotary_validate(ctypes.byref(a)) == _lib.KDA_OK
    a = kda.make_rotary_args(q, k, torch.arange(20), torch.ones(8, dtype=torch.float64), both[:, :4], both[:, 3:5])
    assert lib.kda_rotary_validate(ctypes.byref(a)) == _lib.KDA_ERR_ALIAS
