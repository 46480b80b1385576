"""GPU parity of the norms of q and k with the fp64 oracle, and their gradient with the oracle's and with differences.

Bounds. u is the half step of the tensors' type. In fp32 a row's factor r is within 2^-22 (a root of one unit, a power of two,
a sum in 64 bits), the weight, the product with it and the rotation's two products and sum make 8 more roundings of 2^-24 of
their terms, which are at most sqrt(2) times the row's largest: 2^-20 of the row's largest result, and u of the
element. The gradient's sum over D terms adds D 2^-24 of the terms' sizes, whose sum is at most |u| |x| r <= |u| sqrt(1 / m).
A weight's gradient sums n rows: each term within 2^-20, the sums within sqrt(n) 2^-23 of the terms' root sum square
times sqrt(n), and the result's own half step.
"""
import numpy as np
import pytest
import torch

import gated_delta_rule_pack_amd as kda
from oracle import qk_norm, qk_norm_gradient
from tests.linear_harness import DT, HALF, TINY, f64, same_bits

pytestmark = pytest.mark.gpu

CASES = {
    "plain": dict(),
    "one token": dict(T=1),
    "one head": dict(T=3, Hq=1, Hk=1),
    "no k": dict(Hk=0),
    "l2": dict(kind="l2", weight="none"),
    "l2 weighted": dict(kind="l2", offset=1.0),
    "no rotation": dict(rot=0),
    "part": dict(rot=64),
    "odd part": dict(rot=36),
    "interleaved": dict(interleaved=True),
    "interleaved part": dict(interleaved=True, rot=64),
    "f16": dict(dtype="f16"),
    "f32": dict(dtype="f32"),
    "f32 interleaved": dict(dtype="f32", interleaved=True, rot=40),
    "f32 weights": dict(weight="f32", offset=1.0),
    "no weights": dict(weight="none"),
    "D 64": dict(D=64),
    "D 72": dict(D=72, rot=72),
    "D 80": dict(D=80, rot=40),
    "D 80 whole": dict(D=80, rot=16),
    "D 96": dict(D=96, rot=96, T=50),
    "D 192": dict(D=192, rot=64),
    "D 256 f32": dict(D=256, rot=256, dtype="f32"),
    "D 1": dict(D=1, rot=0),
    "D 5": dict(D=5, rot=2),
    "D 65": dict(D=65, rot=64, dtype="f32"),
    "D 1000": dict(D=1000, rot=0, Hq=2, T=3),
    "D 1024": dict(D=1024, rot=1024, Hq=2, T=3),
    "D 1024 f32": dict(D=1024, rot=512, Hq=2, T=3, dtype="f32", interleaved=True),
    "many": dict(T=2500, Hq=4, Hk=2),
    "many narrow": dict(T=1500, Hq=2, Hk=1, D=36, rot=36),
    "int32 positions": dict(i32=True),
}


def make(T=19, Hq=6, Hk=2, D=128, rot=None, interleaved=False, dtype="bf16", weight="same", offset=0.0, kind="rms", i32=False, seed=3):
    gen = torch.Generator("cpu").manual_seed(seed)
    dt = DT[dtype]
    rot = D if rot is None else rot

    def rows(H):
        return (torch.randn(T, H, D, generator=gen) * torch.exp(torch.randn(T, H, 1, generator=gen))).to(dt) if H else None

    s = dict(q=rows(Hq), k=rows(Hk), gq=rows(Hq), gk=rows(Hk), qw=None, kw=None, pos=None, freq=None)
    if weight != "none":
        wt = dt if weight == "same" else torch.float32
        s["qw"] = (1 - offset + 0.3 * torch.randn(D, generator=gen)).to(wt)
        s["kw"] = (1 - offset + 0.3 * torch.randn(D, generator=gen)).to(wt) if Hk else None
    if rot:
        s["freq"] = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        s["pos"] = torch.randint(0, 100000, (T,), generator=gen).to(torch.int32 if i32 else torch.int64)
    return s, dict(kind=kind, weight_offset=offset, interleaved=interleaved)


def oracle_kw(s, kw):
    return dict(positions=None if s["pos"] is None else f64(s["pos"]), inv_freq=None if s["freq"] is None else f64(s["freq"]),
                l2=kw["kind"] == "l2", offset=kw["weight_offset"], interleaved=kw["interleaved"])


def near(name, got, want, room):
    off = np.abs(got - want)
    assert np.all(np.isfinite(got)), f"{name}: non-finite"
    share = float(np.max(off / np.maximum(room, 1e-300)))
    print(f"  {name}: rel-L2 {np.linalg.norm(off) / max(np.linalg.norm(want), 1e-300):.2e}, worst at {share:.2f} of its bound", flush=True)
    assert share <= 1.0, f"{name}: {share:.3f} of its bound"


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name):
    s, kw = make(**CASES[name])
    d = {n: None if t is None else t.cuda() for n, t in s.items()}
    q, k = kda.qk_norm(d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"], **kw)
    assert (k is None) == (s["k"] is None)
    for n, got, w in (("q", q, "qw"), ("k", k, "kw")):
        if got is None:
            continue
        want = qk_norm(f64(s[n]), None if s[w] is None else f64(s[w]), **oracle_kw(s, kw))
        assert got.dtype == s[n].dtype and got.shape == s[n].shape
        near(n, f64(got), want, HALF[got.dtype] * np.abs(want) + 2.0 ** -20 * np.abs(want).max(-1, keepdims=True) + TINY[got.dtype])


@pytest.mark.parametrize("name", sorted(CASES))
def test_gradient(name):
    s, kw = make(**CASES[name])
    d = {n: None if t is None else t.cuda() for n, t in s.items()}
    dq, dk, dqw, dkw = kda.qk_norm_backward(d["gq"], d["gk"], d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"], **kw)
    for n, got, gotw, w in (("q", dq, dqw, "qw"), ("k", dk, dkw, "kw")):
        if got is None:
            assert s[n] is None and gotw is None
            continue
        x, dy, ok = f64(s[n]), f64(s["g" + n]), oracle_kw(s, kw)
        wide = None if s[w] is None else f64(s[w])
        want, wantw = qk_norm_gradient(dy, x, wide, **ok)
        D, m = x.shape[-1], 1.0 if ok["l2"] else 1.0 / x.shape[-1]
        size = np.sqrt(m * (x * x).sum(-1, keepdims=True) + 1e-6)
        u = np.sqrt((dy * dy).sum(-1, keepdims=True)) * (1.0 if wide is None else np.abs(ok["offset"] + wide).max())
        # The terms z, x m r^2 sum(u x) are at most |u| each (the second's norm too).
        room = HALF[got.dtype] * np.abs(want) + (2.0 ** -20 + D * 2.0 ** -24) * u / size + TINY[got.dtype]
        near("d" + n, f64(got), want, room)
        if wide is None:
            assert gotw is None
            continue
        assert gotw.dtype == s[w].dtype
        y = x / size
        rows = x.shape[0] * x.shape[1]
        terms = np.sqrt(((np.abs(dy).max(-1, keepdims=True) * y) ** 2).sum((0, 1))) * 2 ** 0.5
        near("d" + w, f64(gotw), wantw, HALF[gotw.dtype] * np.abs(wantw) + rows ** 0.5 * (2.0 ** -20 + rows ** 0.5 * 2.0 ** -23) * terms + TINY[gotw.dtype])
