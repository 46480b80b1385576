"""The operators that are measured: linear attention with a decay for each head (prompts and
single tokens, over a dense state or a paged pool) and rotary positions.

Every case is one call as a serving program makes it. ``own`` selects the framework's
kernels; otherwise ``run`` computes the plain form with elementary torch operations.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CHUNK = 128  # tokens per chunk of the plain form


# ---------------------------------------------------------------------------- cases
def listed():
    prefill = dict(op="prefill", n_long=1, n_single=0, seq_seed=0, K=128, V=128, decay="head", resets=False, state="paged",
                   state_dtype="f32", k_first=False, pad=0, fused_qkv=False)
    step = dict(op="step", K=128, V=128, decay="token", state_dtype="f32", k_first=False, rot=0, interleaved=False)
    rot = dict(op="rotary", D=128, rot=128, interleaved=False, dtype="bf16", inverse=False, start=0, stretch=1.0)
    return [
        # A short question to an idle server: launch latency counts.
        dict(prefill, name="prefill_1x37_H12", lo=37, hi=37, H=12, H_qk=12),
        # One prompt at the head count of one GPU.
        dict(prefill, name="prefill_1x4096_H12", lo=4096, hi=4096, H=12, H_qk=12),
        # A long document with decays of its own for each token, some of them resets; padded slots.
        dict(prefill, name="prefill_1x16384_H12_token", lo=16384, hi=16384, H=12, H_qk=12, decay="token", resets=True,
             pad=4096),
        # A full batch of ragged prompts, empty ones among them, over a bf16 pool.
        dict(prefill, name="prefill_128xvar_H12_bf16", n_long=128, lo=0, hi=2048, seq_seed=7, H=12, H_qk=12,
             decay="token", state_dtype="bf16"),
        # Two chunks of prompts beside running requests of one token each, q, k and v rows of one
        # projection's output, narrow value heads that share q and k.
        dict(prefill, name="prefill_mixed_H24_qk4_V64", n_long=2, n_single=62, lo=500, hi=1300, seq_seed=3, H=24, H_qk=4,
             V=64, decay="token", fused_qkv=True),
        # The largest: a book on a model that is not split over GPUs, dense state in and out.
        dict(prefill, name="prefill_1x32768_H32", lo=32768, hi=32768, H=32, H_qk=32, state="dense"),
        # One request's next token.
        dict(step, name="step_1_H12", N=1, H=12, H_qk=12),
        # A full batch of requests over a bf16 pool.
        dict(step, name="step_256_H12_bf16", N=256, H=12, H_qk=12, state_dtype="bf16", decay="head"),
        # A large batch with rotated q and k, shared q/k heads.
        dict(step, name="step_500_H32_qk8_rot", N=500, H=32, H_qk=8, rot=64),
        # Rotation of a few new tokens far into a stretched context.
        dict(rot, name="rotary_7_far", T=7, Hq=32, Hk=8, start=900_000, stretch=8.0),
        # Rotation of a prompt's q and k, half of each head.
        dict(rot, name="rotary_16384_part", T=16384, Hq=32, Hk=8, rot=64),
        # The gradient's rotation back, interleaved pairs, 32-bit gradients.
        dict(rot, name="rotary_5001_back_f32", T=5001, Hq=12, Hk=12, D=64, rot=64, interleaved=True, dtype="f32",
             inverse=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "rotary"])
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 256])
        Hk = rng.choice([1, 2, 4, 8, 12])
        return dict(op=op, T=_log_int(rng, 1, 16384), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, D=D,
                    rot=D if rng.random() < 0.6 else rng.choice([16, 32, D // 2]), interleaved=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), inverse=rng.random() < 0.3,
                    start=rng.choice([0, _log_int(rng, 1, 1_000_000)]), stretch=rng.choice([1.0, 4.0, 32.0]))
    K, V = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (64, 128)])
    H_qk = rng.choice([1, 2, 4, 6, 12])
    H = H_qk * rng.choice([1, 1, 2, 4] if H_qk < 12 else [1, 2])
    both = dict(H=H, H_qk=H_qk, K=K, V=V, decay=rng.choice(["head", "token"]), k_first=rng.random() < 0.3,
                state_dtype=rng.choice(["f32", "f32", "f16", "bf16"]))
    if op == "step":
        return dict(both, op=op, N=_log_int(rng, 1, 512), rot=rng.choice([0, 0, 32, K]), interleaved=rng.random() < 0.5)
    n_long = _log_int(rng, 1, 128)
    hi = _log_int(rng, 16, max(17, min(32768, 1_000_000 // (n_long * H))))  # no more token-heads than the largest listed case
    return dict(both, op=op, n_long=n_long, n_single=rng.choice([0, 0, _log_int(rng, 1, 128)]),
                lo=rng.choice([0, hi // 2, hi]), hi=hi, seq_seed=rng.randrange(1 << 20),
                resets=both["decay"] == "token" and rng.random() < 0.4, state=rng.choice(["paged", "paged", "dense"]),
                pad=rng.choice([0, 0, 64, 4096]), fused_qkv=rng.random() < 0.4)


def _lengths(case):
    """Prompts uniform in [lo, hi], then the single tokens, in an order of their own: the case's, whatever the seed."""
    gen = torch.Generator("cpu").manual_seed(case["seq_seed"])
    lens = torch.randint(case["lo"], case["hi"] + 1, (case["n_long"],), generator=gen).tolist() + [1] * case["n_single"]
    return [lens[i] for i in torch.randperm(len(lens), generator=gen).tolist()]


# ---------------------------------------------------------------------------- inputs
def _decay(case, T, gen, dev):
    """Log decays: one for each head (a geometric series of half-lives), or one for each token and head."""
    H = case["H"]
    if case["decay"] == "head":
        jitter = 1 + 0.05 * torch.rand(H, generator=gen, device=dev)
        return -torch.exp2(-8 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H) * jitter
    x = torch.randn(T, H, generator=gen, device=dev)
    rate = 0.25 + torch.rand(H, generator=gen, device=dev)
    g = -torch.log1p(torch.exp(x - 3)) * rate
    if case.get("resets"):  # a document's end: everything before it is forgotten
        g[torch.rand(T, generator=gen, device=dev) < 1 / 512] = -math.inf
    return g


def _frequencies(rot, stretch, dev):
    """Rotation frequencies of base 10000; ``stretch`` slows all but the fastest (a larger base)."""
    base = 10000.0 * stretch ** (rot / max(rot - 2, 1))
    return base ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)


def _pool(case, slots, pad, gen, dev):
    H, V, K = case["H"], case["V"], case["K"]
    store = torch.empty(slots, H * V * K + pad, device=dev, dtype=DTYPES[case["state_dtype"]])
    store.copy_(torch.randn(store.shape, generator=gen, device=dev))
    planes = (K, V) if case["k_first"] else (V, K)
    return store[:, : H * V * K].unflatten(1, (H, *planes))


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(dev).manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev).to(dtype)

    if case["op"] == "rotary":
        dt = DTYPES[case["dtype"]]
        s = dict(case=case, q=randn(case["T"], case["Hq"], case["D"], dtype=dt), k=randn(case["T"], case["Hk"], case["D"], dtype=dt))
        s["inv_freq"] = _frequencies(case["rot"], case["stretch"], dev)
        s["factor"] = 0.1 * math.log(case["stretch"]) + 1.0
        jump = torch.randint(0, 64, (1,), generator=gen, device=dev)
        s["positions"] = torch.arange(case["T"], device=dev) + case["start"] + jump
        return s
    H, H_qk, K, V = case["H"], case["H_qk"], case["K"], case["V"]
    if case["op"] == "step":
        N = case["N"]
        s = dict(case=case, q=randn(N, H_qk, K), k=randn(N, H_qk, K), v=randn(N, H, V), g=_decay(case, N, gen, dev),
                 scale=K ** -0.5, state_cache=_pool(case, N + N // 8 + 1, 0, gen, dev))
        s["state_indices"] = torch.randperm(N + N // 8 + 1, generator=gen, device=dev)[:N].to(torch.int32)
        s["positions"] = torch.randint(0, 200_000, (N,), generator=gen, device=dev)
        s["inv_freq"] = _frequencies(case["rot"], 1.0, dev) if case["rot"] else None
        return s
    lens = _lengths(case)
    N, T = len(lens), sum(lens)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s = dict(case=case, scale=K ** -0.5, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev),
             cu_seqlens_cpu=torch.tensor(cu, dtype=torch.int32), g=_decay(case, T, gen, dev))
    if case["fused_qkv"]:
        row = randn(T, 2 * H_qk * K + H * V)
        q, k, v = row.split([H_qk * K, H_qk * K, H * V], dim=1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (H_qk, K)), k.unflatten(1, (H_qk, K)), v.unflatten(1, (H, V))
    else:
        s["q"], s["k"], s["v"] = randn(T, H_qk, K), randn(T, H_qk, K), randn(T, H, V)
    if case["state"] == "paged":
        slots = N + 3
        s["state_cache"] = _pool(case, slots, case["pad"], gen, dev)
        s["state_indices"] = torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32)
        s["has_initial_state"] = torch.rand(N, generator=gen, device=dev) < 0.5
    else:
        s["initial_state"] = _pool(case, N, 0, gen, dev)
    # The plain form's plan: the tokens of each chunk, in order, and the sequence that it belongs to.
    per = torch.tensor([-(-n // CHUNK) for n in lens])
    first = torch.cumsum(per, 0) - per
    seq = torch.repeat_interleave(torch.arange(N), per)
    begin = torch.tensor(cu[:-1])[seq] + CHUNK * (torch.arange(len(seq)) - first[seq])
    at = begin[:, None] + torch.arange(CHUNK)
    inside = at < torch.tensor(cu[1:])[seq][:, None]
    some = per > 0
    s["plan"] = dict(tokens=at.clamp(max=max(T - 1, 0)).to(dev), inside=inside.to(dev), seq=seq.to(dev),
                     first=first[seq].to(dev), last=(first + per - 1)[some].to(dev), some=torch.nonzero(some)[:, 0].to(dev))
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    return {"prefill": _prefill, "step": _step, "rotary": _rotary}[s["case"]["op"]](s)


def _prefill(s):
    case = s["case"]
    paged = case["state"] == "paged"
    if own:
        import gated_delta_rule_pack_amd as kda
        state = (dict(state_cache=s["state_cache"], state_indices=s["state_indices"], has_initial_state=s["has_initial_state"])
                 if paged else dict(initial_state=s["initial_state"], output_final_state=True))
        out, final = kda.linear_fwd(s["q"], s["k"], s["v"], s["g"], s["cu_seqlens"], cu_seqlens_cpu=s["cu_seqlens_cpu"],
                                    scale=s["scale"], state_k_first=case["k_first"], **state)
        return {"out": out, "state": s["state_cache"] if paged else final}
    if paged:
        initial = s["state_cache"][s["state_indices"]].float()
        initial = torch.where(s["has_initial_state"][:, None, None, None], initial, torch.zeros_like(initial))
    else:
        initial = s["initial_state"].float()
    out, final = _plain_chunks(s, initial.mT if case["k_first"] else initial)
    final = (final.mT if case["k_first"] else final).to(DTYPES[case["state_dtype"]])
    if paged:
        s["state_cache"][s["state_indices"]] = final
        return {"out": out, "state": s["state_cache"]}
    return {"out": out, "state": final}


def _plain_chunks(s, initial):
    """Chunked form: within a chunk a masked product, across chunks one product with the decays between
    them. Decays are summed in 64 bits; initial and the returned final states are [N, H, V, K]."""
    case, plan = s["case"], s["plan"]
    H, group, V, K = case["H"], case["H"] // case["H_qk"], case["V"], case["K"]
    T = s["q"].shape[0]
    out = torch.empty(T, H, V, dtype=s["v"].dtype, device=s["v"].device)
    if plan["seq"].numel() == 0:
        return out, initial.clone()
    at, inside, seq = plan["tokens"], plan["inside"], plan["seq"]
    nC = at.shape[0]
    here = inside[:, :, None, None]
    q, k = (torch.where(here, s[n][at].float(), 0.0).permute(2, 0, 1, 3).repeat_interleave(group, 0) for n in ("q", "k"))
    v = torch.where(here, s["v"][at].float(), 0.0).permute(2, 0, 1, 3)                       # [H, nC, C, V]
    g = s["g"].double().clamp(min=-1e4)                                                       # e^-10000 is 0
    g = (g[at] if case["decay"] == "token" else g.expand(nC, CHUNK, H)).permute(2, 0, 1)
    G = torch.where(inside, g, 0.0).cumsum(-1)                                                # [H, nC, C]
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=at.device).tril()
    D = torch.where(causal, G[..., :, None] - G[..., None, :], -1e30).float().exp()
    o = ((q @ k.mT) * D) @ v
    local = (v * (G[..., -1:] - G).float().exp()[..., None]).mT @ k                           # [H, nC, V, K]
    before = torch.cat([torch.zeros_like(G[:, :1, -1]), G[..., -1].cumsum(-1)], 1)            # [H, nC + 1]
    order = torch.arange(nC, device=at.device)
    earlier = (order[None, :] < order[:, None]) & (seq[None, :] == seq[:, None])
    M = torch.where(earlier, before[:, :-1, None] - before[:, None, 1:], -1e30).float().exp()  # [H, nC, nC]
    start = (M @ local.flatten(2)).unflatten(2, (V, K))
    from_first = (before[:, :-1] - before[:, :-1].gather(1, plan["first"].expand(H, -1))).float().exp()
    start = start + from_first[..., None, None] * initial[seq].transpose(0, 1)
    o = o + G.float().exp()[..., None] * (q @ start.mT)
    out[at[inside]] = (s["scale"] * o).permute(1, 2, 0, 3)[inside].to(out.dtype)
    final = initial.clone()
    end = G[:, plan["last"], -1].float().exp()[..., None, None] * start[:, plan["last"]] + local[:, plan["last"]]
    final[plan["some"]] = end.transpose(0, 1)
    return out, final


def _step(s):
    case = s["case"]
    if own:
        import gated_delta_rule_pack_amd as kda
        out = kda.linear_step(s["q"], s["k"], s["v"], s["g"], state_cache=s["state_cache"], state_indices=s["state_indices"],
                              scale=s["scale"], state_k_first=case["k_first"], positions=s["positions"] if case["rot"] else None,
                              inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        return {"out": out, "state": s["state_cache"]}
    group = case["H"] // case["H_qk"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if case["rot"]:
        q, k = (_plain_rotation(x, s["positions"], s["inv_freq"], 1.0, case["interleaved"], False) for x in (q, k))
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    S = s["state_cache"][s["state_indices"]].float()
    S = S.mT if case["k_first"] else S
    decay = s["g"].exp().expand(case["N"], -1)[..., None, None]
    S = decay * S + v[..., :, None] * k[..., None, :]
    out = (s["scale"] * (S @ q[..., None])[..., 0]).to(s["v"].dtype)
    s["state_cache"][s["state_indices"]] = (S.mT if case["k_first"] else S).to(s["state_cache"].dtype)
    return {"out": out, "state": s["state_cache"]}


def _rotary(s):
    case = s["case"]
    if own:
        import gated_delta_rule_pack_amd as kda
        q, k = kda.rotary(s["q"], s["k"], s["positions"], s["inv_freq"], interleaved=case["interleaved"],
                          factor=s["factor"], inverse=case["inverse"])
        return {"q": q, "k": k}
    return {n: _plain_rotation(s[n].float(), s["positions"], s["inv_freq"], s["factor"], case["interleaved"],
                               case["inverse"]).to(s[n].dtype) for n in ("q", "k")}


def _plain_rotation(x, positions, inv_freq, factor, interleaved, inverse):
    """x [T, H, D] in 32 bits, its first 2 * len(inv_freq) channels rotated; angles in 64 bits."""
    half = inv_freq.numel()
    angle = (positions.double()[:, None] * inv_freq)[:, None]
    c, n = (factor * angle.cos()).float(), (factor * (-angle if inverse else angle).sin()).float()
    x, rest = x[..., : 2 * half], x[..., 2 * half :]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    pair = (a * c - b * n, a * n + b * c)
    return torch.cat([torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1), rest], -1)


# ---------------------------------------------------------------------------- what a pass can not do without
def work(case):
    if case["op"] == "rotary":
        es = 4 if case["dtype"] == "f32" else 2
        rows = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": 2 * rows * case["D"] * es + 8 * case["T"] + 4 * case["rot"], "flops": 3 * rows * case["rot"]}
    H, H_qk, K, V = case["H"], case["H_qk"], case["K"], case["V"]
    es = 4 if case["state_dtype"] == "f32" else 2
    if case["op"] == "step":
        T = N = case["N"]
        planes = 2 * N
    else:
        lens = _lengths(case)
        T, N = sum(lens), len(lens)
        planes = (1.5 if case["state"] == "paged" else 2) * N  # half of the pool's slots hold a state
    tokens = T * 2 * (2 * H_qk * K + 2 * H * V) + 4 * H * (T if case["decay"] == "token" else 1)
    return {"bytes": tokens + planes * H * V * K * es, "flops": 4 * T * H * K * V}


# ---------------------------------------------------------------------------- 64 bits, from the definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return {n: _turn(s[n], s["positions"], s["inv_freq"], s["factor"], case) for n in ("q", "k")}
    group = case["H"] // case["H_qk"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if case["op"] == "step":
        if case["rot"]:
            turn = dict(case, inverse=False)
            q, k = _turn(q, s["positions"], s["inv_freq"], 1.0, turn), _turn(k, s["positions"], s["inv_freq"], 1.0, turn)
        begin = list(range(case["N"]))
        lens = [1] * case["N"]
    else:
        cu = s["cu_seqlens_cpu"].tolist()
        begin, lens = cu[:-1], [b - a for a, b in zip(cu, cu[1:])]
    lam = torch.exp(s["g"].double())
    lam = lam if case["decay"] == "token" else lam.expand(q.shape[0], -1)
    if "initial_state" in s:
        S = s["initial_state"].double()
    else:
        slots = s["state_indices"].long()
        S = s["state_cache"][slots].double()
        if "has_initial_state" in s:
            S = S * s["has_initial_state"].double()[:, None, None, None]
    S = S.transpose(-1, -2).contiguous() if case["k_first"] else S.contiguous()
    # One token of every sequence at a time, the longest sequences first.
    order = sorted(range(len(lens)), key=lambda n: -lens[n])
    where = torch.tensor(order, device=S.device)
    S, start = S[where], torch.tensor(begin, device=S.device)[where]
    out = torch.empty(v.shape, dtype=torch.float64, device=v.device)
    left = len(order)
    for t in range(max(lens)):
        while left and lens[order[left - 1]] <= t:
            left -= 1
        row, live = start[:left] + t, S[:left]
        kt, qt = k[row].repeat_interleave(group, 1), q[row].repeat_interleave(group, 1)
        live.mul_(lam[row][:, :, None, None]).addcmul_(v[row][..., None], kt[:, :, None, :])
        out[row] = (live * qt[:, :, None, :]).sum(-1)
    back = torch.empty_like(S)
    back[where] = S
    back = back.transpose(-1, -2) if case["k_first"] else back
    if "initial_state" in s:
        return {"out": out * s["scale"], "state": back}
    pool = s["state_cache"].double()
    pool[slots] = back
    return {"out": out * s["scale"], "state": pool}


def _turn(x, positions, inv_freq, factor, case):
    """The rotation as a product with complex numbers."""
    half = inv_freq.numel()
    x = x.double()
    head, rest = x[..., : 2 * half], x[..., 2 * half :]
    pairs = head.unflatten(-1, (half, 2)) if case["interleaved"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
    angle = positions.double()[:, None] * inv_freq
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, factor), -angle if case["inverse"] else angle)[:, None]
    pairs = torch.view_as_real(z)
    head = pairs.flatten(-2) if case["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
    return torch.cat([head, rest], -1)
