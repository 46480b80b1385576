"""Inputs, calls and error bounds of the gated delta rule's tests.

Both sides take the same stored bits. A step S <- S (I - beta k k^T) + ... with 0 <= beta |k|^2 <= 2 never enlarges a row
of S, nor an error that a row already has, so what a token's roundings do to a row is the row's error in the end at most,
and independent roundings of n tokens add up as sqrt(n).

With M the largest value among a sequence's values and states, e2 = 2^-20 what two fp16 terms leave of a channel's largest
operand (2^-21) together with fp32's own roundings of the sums they go into, and e1 = 2^-11 what one term leaves:

* four operands are rounded on a token's way into the state (S, T, what is to be learnt, D): its injection is at most
  4 e M in norm (beta |k| <= sqrt(2 beta) is taken as 1; sums of K independent roundings e of k_j S_j make e |k|), so a
  state element of a sequence of n tokens is off by at most 4 e M (1 + sqrt n), and rounded to its own type;
* decays: exponentials are within (2 + |x|) 2^-24 with |x| <= 120, but a factor e^x multiplies its argument's error away:
  x e^x <= 1; three of them a token stay below 2^-21 M, inside e2;
* an output is scale S q, of a state and q's products in one term (4 e1 M |q|), the state's own error times |q|, and its
  own type's half step.

Single tokens are fp32 throughout: K 2^-24 M for each of three sums of K products, below 2^-15 M in all with K = 128.
"""
from __future__ import annotations

import numpy as np
import torch

import gated_delta_rule_pack_amd as kda
from oracle import delta_forward
from tests.linear_harness import DT, HALF, TINY, Case, f64, same_bits

E1, E2, STEP = 2.0 ** -11, 2.0 ** -20, 2.0 ** -15


class DeltaCase(Case):
    """A linear case's inputs with step sizes; unit: q and k of unit length but for their rounding, else the call
    normalises them."""

    def __init__(self, lengths, H=2, *, dtype="bf16", beta_dtype="f32", unit=False, beta_max=1.0, seed=0, **kw):
        super().__init__(lengths, H, seed=seed, **kw)
        gen = torch.Generator("cpu").manual_seed(seed + 7919)
        self.dtype, self.normalize = DT[dtype], not unit
        q, k = self.q.float(), self.k.float()
        if unit:
            q, k = (x / x.norm(dim=-1, keepdim=True).clamp(min=1e-9) for x in (q, k))
        if self.row is not None:
            self.row = torch.cat([q.flatten(1), k.flatten(1), self.v.float().flatten(1)], 1).to(self.dtype)
            q, k, v = self.row.split([self.H_qk * self.K, self.H_qk * self.K, self.H * self.V], 1)
            self.q, self.k = q.unflatten(1, (self.H_qk, self.K)), k.unflatten(1, (self.H_qk, self.K))
            self.v = v.unflatten(1, (self.H, self.V))
        else:
            self.q, self.k, self.v = q.to(self.dtype), k.to(self.dtype), self.v.to(self.dtype)
        self.beta = (beta_max * torch.randn(self.T, self.H, generator=gen).sigmoid()).to(DT[beta_dtype])

    def oracle(self):
        g = None if self.g is None else f64(self.g)
        return delta_forward(f64(self.q), f64(self.k), f64(self.v), g, f64(self.beta), self.cu.tolist(), scale=self.scale,
                             initial=self.start(), normalize=self.normalize)

    def device(self, dev="cuda"):
        d = super().device(dev)
        d["beta"] = self.beta.to(dev)
        return d

    def forward(self, d, **kw):
        state = {}
        if self.state == "dense":
            state = dict(initial_state=d["initial"], output_final_state=True)
        elif self.state == "paged":
            state = dict(state_cache=d["cache"], state_indices=d["indices"], has_initial_state=d["flags"])
        kw = {**state, **dict(scale=self.scale, state_k_first=self.k_first, normalize=self.normalize), **kw}
        return kda.gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"], **kw)

    def step(self, d, **kw):
        kw = {**dict(state_cache=d["cache"], state_indices=d["indices"], has_initial_state=d["flags"], scale=self.scale,
                     state_k_first=self.k_first, normalize=self.normalize), **kw}
        return kda.gated_delta_step(d["q"], d["k"], d["v"], d["g"], d["beta"], **kw)

    def query_size(self):
        """|q| as the rule takes it, [T, H, 1]."""
        q = f64(self.q)
        if self.normalize:
            return np.ones((self.T, self.H, 1))
        return np.repeat(np.sqrt((q * q).sum(-1, keepdims=True)), self.H // self.H_qk, axis=1)


def close(name, got, want, room):
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.all(np.isfinite(got)), f"{name}: non-finite"
    off = np.abs(got - want)
    norm = np.linalg.norm(want)
    rel = np.linalg.norm(off) / norm if norm else np.linalg.norm(off)
    share = float(np.max(off / np.maximum(room, 1e-300))) if off.size else 0.0
    print(f"  {name}: rel-L2 {rel:.2e}, worst element at {share:.2f} of its bound", flush=True)
    assert share <= 1.0, f"{name}: an element is off by {share:.3f} of its bound"
    return rel


def check(case, out, d, final, step=False):
    """Outputs and final states of one call against the oracle. Rows behind the last bound are not looked at."""
    o, S, size = case.oracle()
    rows = int(case.cu[-1])
    sdt = None if case.state == "none" else (case.initial if case.state == "dense" else case.store).dtype
    one = case.state == "none" or sdt == torch.bfloat16
    n = np.maximum(np.array(case.lengths, np.float64), 1)[:, None]
    state_off = (STEP if step else 4 * (E1 if one else E2) * (1 + np.sqrt(n))) * size         # [N, H]
    token_off = np.repeat(state_off + (0 if step else 4 * E1) * size, case.lengths, axis=0)   # [rows, H]
    u = HALF[case.dtype]
    room = u * np.abs(o[:rows]) + (1 + u) * case.scale * case.query_size()[:rows] * token_off[:, :, None] + TINY[case.dtype]
    rel = close("out", f64(out).reshape(o.shape)[:rows], o[:rows], room)
    # Its own rounding is at most u and averages u / sqrt(3); what one fp16 term leaves of four operands is 4 e1 / sqrt(3).
    assert rows * case.H < 64 or rel < 1.1 * (u + 4 * E1) / 3 ** 0.5, f"out: rel-L2 {rel:.2e}"
    if case.state != "none":
        got = case.finals(d, final)
        kept = ~np.isnan(got).all(axis=(1, 2, 3))
        assert kept.sum() == sum(1 for i in (case.indices.tolist() if case.state == "paged" else range(case.N))
                                 if case.state == "dense" or 0 <= i < case.slots)
        empty = np.array(case.lengths)[:, None] == 0  # read and written back
        room = HALF[sdt] * np.abs(S) + ((1 + HALF[sdt]) * np.where(empty, 0, state_off))[:, :, None, None] + TINY[sdt]
        rel = close("state", got[kept], S[kept], room[kept])
        assert sdt != torch.float32 or rel < 3e-6, f"state: rel-L2 {rel:.2e}"


__all__ = ["DeltaCase", "check", "close", "same_bits", "f64", "DT", "HALF", "TINY"]
