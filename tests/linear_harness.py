"""Inputs, calls and error bounds of the linear-attention and rotary tests.

Both sides take the same stored bits. u = 2^-8 is the half step of bf16 relative to the value
(fp16 2^-11, fp32 2^-24). With A the sums of the terms' absolute values, from the oracle on the
inputs' absolute values:

* an output is rounded three times at most: P or the state for its product (each at most u of its
  terms, together at most u A), and the result (u |o|);
* the fp32 sums and exponentials stay below EPS32 A for states and outputs alike: a sum of n terms is
  off by at most n 2^-24 of A in any order, a chunked sum of 64 tokens in three terms by less than
  192 2^-24, and every later chunk adds its own product with e^{G_C} and its sum, three roundings
  more each; an exponential is within (2 + |x|) 2^-24 of e^x, with |x| <= 104 before it is 0, and
  there are at most two in a factor; decays that multiply the older terms shrink their errors too;
* a stored fp16 or bf16 state adds its half step.
"""
from __future__ import annotations

import numpy as np
import torch

import gated_delta_rule_pack_amd as kda
from oracle import linear_forward, rotate

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def eps32(longest):
    """EPS32 for sequences of at most ``longest`` tokens."""
    return 2.0 ** -24 * (192 + 212 + 3 * (longest // 64 + 2))


def f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """One call's inputs, drawn on the CPU from a seed."""

    def __init__(self, lengths, H=2, H_qk=None, K=128, V=128, *, seed=0, decay="token", g_dtype="f32", state="paged",
                 state_dtype="f32", k_first=False, pad=0, extra_rows=0, fused=False, flags="some", tail=0.0, slots=None):
        gen = torch.Generator("cpu").manual_seed(seed)
        self.lengths, self.H, self.K, self.V = list(lengths), H, K, V
        self.H_qk = H_qk or H
        self.k_first, self.state, self.scale = k_first, state, K ** -0.5
        N = len(self.lengths)
        cu = np.concatenate([[0], np.cumsum(self.lengths)]).astype(np.int32)
        self.cu = torch.from_numpy(cu)
        T = int(cu[-1]) + extra_rows
        self.T, self.N = T, N

        def randn(*shape):
            return torch.randn(shape, generator=gen)

        if fused:
            row = randn(T, 2 * self.H_qk * K + H * V).bfloat16()
            q, k, v = row.split([self.H_qk * K, self.H_qk * K, H * V], 1)
            self.row = row
            self.q, self.k, self.v = q.unflatten(1, (self.H_qk, K)), k.unflatten(1, (self.H_qk, K)), v.unflatten(1, (H, V))
        else:
            self.q, self.k, self.v = (randn(T, h, d).bfloat16() for h, d in ((self.H_qk, K), (self.H_qk, K), (H, V)))
            self.row = None
        if decay == "none":
            self.g = None
        elif decay == "head":
            self.g = -torch.exp(randn(H) - 2)
        elif decay == "growth":
            self.g = 0.05 * randn(T, H)
        else:
            self.g = -torch.exp(randn(T, H) - 2)
            if decay == "resets":
                self.g[torch.rand(T, H, generator=gen) < 0.05] = -float("inf")
                self.g[torch.rand(T, H, generator=gen) < 0.05] = -80.0
                self.g[torch.rand(T, H, generator=gen) < 0.05] = float(torch.finfo(torch.float32).min)
        if self.g is not None:
            self.g = self.g.to(DT[g_dtype])
        sdt = DT[state_dtype]
        planes = (K, V) if k_first else (V, K)
        self.initial = self.store = self.indices = self.flags = None
        self.stride0 = H * K * V + pad
        if state == "dense":
            self.initial = (randn(N, H, *planes) * 0.5).to(sdt)
        elif state == "paged":
            slots = slots or N + 2
            self.slots = slots
            self.store = (randn(slots, self.stride0) * 0.5).to(sdt)
            self.indices = torch.randperm(slots, generator=gen)[:N].to(torch.int32)
            self.flags = {"some": torch.rand(N, generator=gen) < 0.5, "all": torch.ones(N, dtype=torch.bool)}[flags]
            for n in range(N):
                if not self.flags[n]:
                    self.store[int(self.indices[n]), : H * K * V] = float("nan")  # must not be read
            if pad:
                self.store[:, H * K * V:] = float("nan")

    def planes(self, flat):
        K, V = self.K, self.V
        return flat[:, : self.H * K * V].unflatten(1, (self.H, *((K, V) if self.k_first else (V, K))))

    def start(self):
        """The initial states as [N, H, V, K] in fp64."""
        if self.state == "none":
            return None
        if self.state == "dense":
            S = f64(self.initial)
        else:
            S = np.zeros((self.N, self.H, *self.planes(self.store).shape[2:]))
            for n in range(self.N):
                i = int(self.indices[n])
                if self.flags[n] and 0 <= i < self.slots:
                    S[n] = f64(self.planes(self.store)[i])
        return S.swapaxes(-1, -2) if self.k_first else S

    def oracle(self, q=None, k=None):
        """(out, |out| bound sums, final, |final| bound sums), fp64."""
        g = None if self.g is None else f64(self.g)
        q, k = f64(self.q) if q is None else q, f64(self.k) if k is None else k
        a = (q, k, f64(self.v), g, self.cu.tolist())
        kw = dict(scale=self.scale, initial=self.start())
        return (*linear_forward(*a, **kw), *linear_forward(*a, **kw, absolute=True))

    def device(self, dev="cuda"):
        d = {n: getattr(self, n).to(dev) for n in ("q", "k", "v") if self.row is None}
        if self.row is not None:
            row = self.row.to(dev)
            q, k, v = row.split([self.H_qk * self.K, self.H_qk * self.K, self.H * self.V], 1)
            d = dict(q=q.unflatten(1, (self.H_qk, self.K)), k=k.unflatten(1, (self.H_qk, self.K)), v=v.unflatten(1, (self.H, self.V)))
        d["g"] = None if self.g is None else self.g.to(dev)
        d["cu"] = self.cu.to(dev)
        if self.state == "dense":
            d["initial"] = self.initial.to(dev)
        elif self.state == "paged":
            d["store"] = self.store.to(dev)
            d["cache"] = self.planes(d["store"])
            d["indices"], d["flags"] = self.indices.to(dev), self.flags.to(dev)
        return d

    def forward(self, d, **kw):
        state = {}
        if self.state == "dense":
            state = dict(initial_state=d["initial"], output_final_state=True)
        elif self.state == "paged":
            state = dict(state_cache=d["cache"], state_indices=d["indices"], has_initial_state=d["flags"])
        kw = {**state, **dict(scale=self.scale, state_k_first=self.k_first), **kw}
        return kda.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], **kw)

    def finals(self, d, final):
        """The final states the device holds, [N, H, V, K] fp64, NaN for sequences without a slot."""
        if self.state == "dense":
            S = f64(final)
        else:
            cache = f64(self.planes(d["store"]))
            S = np.stack([cache[int(i)] if 0 <= int(i) < self.slots else np.full(cache.shape[1:], np.nan) for i in self.indices])
        return S.swapaxes(-1, -2) if self.k_first else S


def close(name, got, want, sums, half, longest, own_half, tiny=0.0):
    """|got - want| <= (half + EPS32) sums + own_half |want|, elementwise; prints the worst share of it."""
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{name}: non-finite"
    room = (half + eps32(longest)) * sums * (1 + own_half) + own_half * np.abs(want) + tiny
    off = np.abs(got - want)
    norm = np.linalg.norm(want)
    rel = np.linalg.norm(off) / norm if norm else np.linalg.norm(off)
    share = float(np.max(off / np.maximum(room, 1e-300))) if off.size else 0.0
    print(f"  {name}: rel-L2 {rel:.2e}, worst element at {share:.2f} of its bound", flush=True)
    assert share <= 1.0, f"{name}: an element is off by {share:.3f} of its bound"
    return rel


def check(case, out, d, final, q=None, k=None, extra=0.0, extra_state=0.0):
    """Outputs and final states of one prompt call against the oracle. extra, extra_state: bounds of
    further roundings relative to the terms' sizes. Rows behind the last bound are not looked at."""
    o, S, oa, Sa = case.oracle(q, k)
    longest = max(case.lengths + [1])
    rows = int(case.cu[-1])
    u = HALF[torch.bfloat16]
    rel = close("out", f64(out).reshape(o.shape)[:rows], o[:rows], oa[:rows], u + extra, longest, u, TINY[torch.bfloat16])
    # Independent roundings of at most u each, two of them, average to u / sqrt(3) each: 3.2e-3.
    assert extra or rows * case.H < 64 or rel < 4e-3, f"out: rel-L2 {rel:.2e}"
    if case.state != "none":
        sdt = (case.initial if case.state == "dense" else case.store).dtype
        got = case.finals(d, final)
        kept = ~np.isnan(got).all(axis=(1, 2, 3))
        assert kept.sum() == sum(1 for i in (case.indices.tolist() if case.state == "paged" else range(case.N))
                                 if case.state == "dense" or 0 <= i < case.slots)
        close("state", got[kept], S[kept], Sa[kept], extra_state, longest, HALF[sdt], TINY[sdt])


def same_bits(a, b):
    w = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return torch.equal(a.contiguous().view(w), b.contiguous().view(w))


__all__ = ["Case", "check", "close", "same_bits", "rotate", "f64", "DT", "HALF", "TINY", "eps32"]
