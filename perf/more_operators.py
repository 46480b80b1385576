"""More measured operators: the gated delta rule with one decay for each head (prompts and single
tokens, over a dense state or a paged pool), and the norms of q and k for each head with the position
rotation in the same pass, with their gradient.

Every case is one call as a serving or training program makes it. ``own`` selects the framework's
kernels; otherwise ``run`` computes the plain form with elementary torch operations.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CHUNK = 64  # tokens per chunk of the plain form
EPS = 1e-6


# ---------------------------------------------------------------------------- cases
def listed():
    prompts = dict(op="prompts", n_long=1, n_single=0, seq_seed=0, K=128, V=128, decay="token", resets=False, beta="f32",
                   normalize=True, state="paged", state_dtype="f32", k_first=False, pad=0, fused_qkv=False, dtype="bf16")
    step = dict(op="step", K=128, V=128, decay="token", beta="f32", normalize=True, state_dtype="f32", k_first=False, dtype="bf16")
    norm = dict(op="norm", D=128, rot=128, interleaved=False, dtype="bf16", weight="same", offset=0.0, kind="rms", start=0)
    return [
        # A short question to an idle server: launch latency counts.
        dict(prompts, name="delta_1x37_H12", lo=37, hi=37, H=12, H_qk=12),
        # One prompt at the head count of one GPU.
        dict(prompts, name="delta_1x4096_H12", lo=4096, hi=4096, H=12, H_qk=12),
        # A long document of which some tokens forget everything before them; q and k already of unit length,
        # padded slots.
        dict(prompts, name="delta_1x16384_H12_unit", lo=16384, hi=16384, H=12, H_qk=12, resets=True, normalize=False, pad=4096),
        # A full batch of ragged prompts, empty ones among them, over a bf16 pool.
        dict(prompts, name="delta_128xvar_H12_bf16", n_long=128, lo=0, hi=2048, seq_seed=7, H=12, H_qk=12, state_dtype="bf16"),
        # Prompts beside running requests of one token each, q, k and v rows of one projection's output, narrow
        # value heads that share q and k, fp16.
        dict(prompts, name="delta_mixed_H24_qk4_V64_f16", n_long=2, n_single=62, lo=500, hi=1300, seq_seed=3, H=24, H_qk=4,
             V=64, fused_qkv=True, dtype="f16"),
        # The largest: a book on a model that is not split over GPUs, pairs of value heads, dense state in and out.
        dict(prompts, name="delta_1x32768_H32_qk16", lo=32768, hi=32768, H=32, H_qk=16, state="dense"),
        # One request's next token.
        dict(step, name="delta_step_1_H12", N=1, H=12, H_qk=12),
        # A full batch of requests over a bf16 pool, heads that share q and k.
        dict(step, name="delta_step_300_H32_qk16_bf16", N=300, H=32, H_qk=16, state_dtype="bf16", beta="bf16"),
        # q and k of a few new tokens far into a context.
        dict(norm, name="norm_7_far", back=False, T=7, Hq=32, Hk=8, start=900_000, offset=1.0),
        # q and k of a long prompt, half of each head rotated.
        dict(norm, name="norm_16384_part", back=False, T=16384, Hq=32, Hk=8, rot=64),
        # The gradient over a batch of training sequences.
        dict(norm, name="norm_back_8192", back=True, T=8192, Hq=32, Hk=8, weight="f32"),
        # The gradient in 32 bits, interleaved pairs, heads of an odd size.
        dict(norm, name="norm_back_1001_f32_D72", back=True, T=1001, Hq=12, Hk=12, D=72, rot=36, interleaved=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompts", "prompts", "prompts", "step", "norm", "norm"])
    if op == "norm":
        D = rng.choice([64, 72, 80, 96, 128, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8, 12])
        return dict(op=op, back=rng.random() < 0.5, T=_log_int(rng, 1, 16384), Hq=Hk * rng.choice([1, 2, 4]), Hk=Hk, D=D,
                    rot=rng.choice([0, D, D, 32, D // 2]), interleaved=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), weight=rng.choice(["same", "f32", "none"]),
                    offset=rng.choice([0.0, 1.0]), kind=rng.choice(["rms", "rms", "l2"]),
                    start=rng.choice([0, _log_int(rng, 1, 1_000_000)]))
    K, V = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (64, 128)])
    H_qk = rng.choice([1, 2, 4, 6, 12])
    H = H_qk * rng.choice([1, 1, 2, 4] if H_qk < 12 else [1, 2])
    both = dict(H=H, H_qk=H_qk, K=K, V=V, decay=rng.choice(["token", "token", "head", "none"]), beta=rng.choice(["f32", "bf16"]),
                normalize=rng.random() < 0.7, k_first=rng.random() < 0.3, state_dtype=rng.choice(["f32", "f32", "f16", "bf16"]),
                dtype=rng.choice(["bf16", "bf16", "f16"]))
    if op == "step":
        return dict(both, op=op, N=_log_int(rng, 1, 512))
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
    """Log decays: none, one for each head (a geometric series of half-lives), or one for each token and head (a rate
    of the head times a step size of the token, as selective models make them)."""
    H = case["H"]
    if case["decay"] == "none":
        return None
    if case["decay"] == "head":
        jitter = 1 + 0.05 * torch.rand(H, generator=gen, device=dev)
        return -torch.exp2(-8 * torch.arange(1, H + 1, device=dev, dtype=torch.float32) / H) * jitter
    x = torch.randn(T, H, generator=gen, device=dev)
    rate = 0.5 + 15.5 * torch.rand(H, generator=gen, device=dev)
    size = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(H, generator=gen, device=dev))
    g = -rate * torch.log1p(torch.exp(x + size.expm1().log()))
    if case.get("resets"):  # a document's end: everything before it is forgotten
        g[torch.rand(T, generator=gen, device=dev) < 1 / 512] = -math.inf
    return g


def _pool(case, slots, pad, gen, dev):
    H, V, K = case["H"], case["V"], case["K"]
    store = torch.empty(slots, H * V * K + pad, device=dev, dtype=DTYPES[case["state_dtype"]])
    store.copy_(0.3 * torch.randn(store.shape, generator=gen, device=dev))
    planes = (K, V) if case["k_first"] else (V, K)
    return store[:, : H * V * K].unflatten(1, (H, *planes))


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    if case["op"] == "norm":
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        s = dict(case=case, q=(1.5 * randn(T, Hq, D)).to(dt), k=(1.5 * randn(T, Hk, D)).to(dt), q_weight=None, k_weight=None)
        if case["weight"] != "none":
            wt = dt if case["weight"] == "same" else torch.float32
            s["q_weight"], s["k_weight"] = ((1 - case["offset"] + 0.2 * randn(D)).to(wt) for _ in range(2))
        if case["back"]:
            s["grad_q"], s["grad_k"] = randn(T, Hq, D).to(dt), randn(T, Hk, D).to(dt)
        s["positions"] = s["inv_freq"] = None
        if case["rot"]:
            s["inv_freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
            s["positions"] = torch.arange(T, device=dev) + case["start"] + torch.randint(0, 64, (1,), generator=gen, device=dev)
        return s
    H, H_qk, K, V = case["H"], case["H_qk"], case["K"], case["V"]
    lens = [1] * case["N"] if case["op"] == "step" else _lengths(case)
    N, T = len(lens), sum(lens)
    q, k, v = randn(T, H_qk, K), randn(T, H_qk, K), randn(T, H, V)
    if not case["normalize"]:  # of unit length up to their type's rounding
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    s = dict(case=case, scale=K ** -0.5, g=_decay(case, T, gen, dev), beta=randn(T, H).sigmoid().to(DTYPES[case["beta"]]))
    if case.get("fused_qkv"):
        row = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).to(dt)
        q, k, v = row.split([H_qk * K, H_qk * K, H * V], dim=1)
        s["q"], s["k"], s["v"] = q.unflatten(1, (H_qk, K)), k.unflatten(1, (H_qk, K)), v.unflatten(1, (H, V))
    else:
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), v.to(dt)
    if case["op"] == "step":
        slots = N + N // 8 + 1
        s["state_cache"] = _pool(case, slots, 0, gen, dev)
        s["state_indices"] = torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32)
        return s
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    s["cu_seqlens_cpu"] = torch.tensor(cu, dtype=torch.int32)
    if case["state"] == "paged":
        slots = N + 3
        s["state_cache"] = _pool(case, slots, case["pad"], gen, dev)
        s["state_indices"] = torch.randperm(slots, generator=gen, device=dev)[:N].to(torch.int32)
        s["has_initial_state"] = torch.rand(N, generator=gen, device=dev) < 0.5
    else:
        s["initial_state"] = _pool(case, N, 0, gen, dev)
    # The plain form's plan: the tokens of each chunk, in order, the sequence that it belongs to, the first chunk of a
    # sequence, and for sequences with tokens their last chunk.
    per = torch.tensor([-(-n // CHUNK) for n in lens])
    first = torch.cumsum(per, 0) - per
    seq = torch.repeat_interleave(torch.arange(N), per)
    place = torch.arange(len(seq)) - first[seq]
    at = torch.tensor(cu[:-1])[seq][:, None] + CHUNK * place[:, None] + torch.arange(CHUNK)
    inside = at < torch.tensor(cu[1:])[seq][:, None]
    some = per > 0
    s["plan"] = dict(tokens=at.clamp(max=max(T - 1, 0)).to(dev), inside=inside.to(dev), seq=seq.to(dev), begins=(place == 0).to(dev),
                     last=(first + per - 1)[some].to(dev), some=torch.nonzero(some)[:, 0].to(dev),
                     longest=int(per.max()) if N else 0)
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    return {"prompts": _prompts, "step": _step, "norm": _norm}[s["case"]["op"]](s)


def _prompts(s):
    case = s["case"]
    paged = case["state"] == "paged"
    if own:
        import gated_delta_rule_pack_amd as kda
        state = (dict(state_cache=s["state_cache"], state_indices=s["state_indices"], has_initial_state=s["has_initial_state"])
                 if paged else dict(initial_state=s["initial_state"], output_final_state=True))
        out, final = kda.gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu_seqlens"],
                                         cu_seqlens_cpu=s["cu_seqlens_cpu"], scale=s["scale"], normalize=case["normalize"],
                                         state_k_first=case["k_first"], **state)
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


def _unit(x):
    return x * (x.square().sum(-1, keepdim=True) + EPS).rsqrt()


def _plain_chunks(s, initial):
    """Chunked form. Within a chunk the rule is a triangular system, solved by halves; a chunk takes the state S
    to S A + B, and the chunks' maps are composed by doubling. Decays are summed in 64 bits; initial and the returned final
    states are [N, H, V, K]."""
    case, plan = s["case"], s["plan"]
    H, group, V, K = case["H"], case["H"] // case["H_qk"], case["V"], case["K"]
    T = s["q"].shape[0]
    out = torch.empty(T, H, V, dtype=s["v"].dtype, device=s["v"].device)
    if plan["seq"].numel() == 0:
        return out, initial.clone()
    at, inside, seq = plan["tokens"], plan["inside"], plan["seq"]
    n, C = at.shape
    here = inside[:, :, None, None]
    q, k = (s[x].float() for x in ("q", "k"))
    q, k = (_unit(q), _unit(k)) if case["normalize"] else (q, k)
    q, k = (torch.where(here, x[at], 0.0).permute(2, 0, 1, 3).repeat_interleave(group, 0) for x in (q, k))  # [H, n, C, K]
    v = torch.where(here, s["v"][at].float(), 0.0).permute(2, 0, 1, 3)                                      # [H, n, C, V]
    beta = torch.where(inside[:, :, None], s["beta"][at].float(), 0.0).permute(2, 0, 1)                     # [H, n, C]
    if s["g"] is None:
        G = torch.zeros(H, n, C, dtype=torch.float64, device=at.device)
    else:
        g = s["g"].double().clamp(min=-1e4)                                                                # e^-10000 is 0
        g = (g[at] if case["decay"] == "token" else g.expand(n, C, H)).permute(2, 0, 1)
        G = torch.where(inside, g, 0.0).cumsum(-1)
    causal = torch.ones(C, C, dtype=torch.bool, device=at.device).tril()
    D = torch.where(causal, G[..., :, None] - G[..., None, :], -1e30).float().exp()
    A = beta[..., None] * (k @ k.mT) * D * causal.tril(-1)
    inverse = torch.eye(C, device=at.device).expand(H, n, C, C).clone()
    b = 1
    while b < C:  # the inverse of I + A: of two diagonal blocks X and Y and the block A' below X, -Y A' X stands below X
        low, X, Y = (_blocks(m, b, i, j) for m, i, j in ((A, 1, 0), (inverse, 0, 0), (inverse, 1, 1)))
        _blocks(inverse, b, 1, 0).copy_(-(Y @ low @ X))
        b *= 2
    W = inverse @ (k * (beta * G.float().exp())[..., None])
    U = inverse @ (v * beta[..., None])
    end = G[..., -1:]
    left = k * (end - G).float().exp()[..., None]
    begins = plan["begins"][None, :, None, None]
    # S -> S move + add; where a sequence begins its initial state goes into add.
    move = end.float().exp()[..., None] * torch.eye(K, device=at.device) - W.mT @ left
    add = U.mT @ left
    start = initial[seq].transpose(0, 1)
    add = add + torch.where(begins, start @ move, 0.0)
    move = torch.where(begins, 0.0, move)
    d = 1
    while d < plan["longest"]:
        add = torch.cat([add[:, :d], add[:, :-d] @ move[:, d:] + add[:, d:]], 1)
        move = torch.cat([move[:, :d], move[:, :-d] @ move[:, d:]], 1)
        d *= 2
    before = torch.where(begins, start, torch.cat([add[:, :1], add[:, :-1]], 1))                           # [H, n, V, K]
    delta = U - W @ before.mT
    o = G.float().exp()[..., None] * (q @ before.mT) + ((q @ k.mT) * D) @ delta
    out[at[inside]] = (s["scale"] * o).permute(1, 2, 0, 3)[inside].to(out.dtype)
    final = initial.clone()
    final[plan["some"]] = add[:, plan["last"]].transpose(0, 1)
    return out, final


def _blocks(m, b, i, j):
    """Of each diagonal block of 2b rows of the last two dimensions its part (i, j) of b rows, as a view."""
    lead, C = m.shape[:-2], m.shape[-1]
    pairs = m.view(*lead, C // (2 * b), 2 * b, C // (2 * b), 2 * b).diagonal(dim1=-4, dim2=-2).movedim(-1, -3)
    return pairs[..., i * b : (i + 1) * b, j * b : (j + 1) * b]


def _step(s):
    case = s["case"]
    if own:
        import gated_delta_rule_pack_amd as kda
        out = kda.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], state_cache=s["state_cache"],
                                   state_indices=s["state_indices"], scale=s["scale"], normalize=case["normalize"],
                                   state_k_first=case["k_first"])
        return {"out": out, "state": s["state_cache"]}
    group = case["H"] // case["H_qk"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    q, k = (_unit(q), _unit(k)) if case["normalize"] else (q, k)
    q, k = q.repeat_interleave(group, 1), k.repeat_interleave(group, 1)
    S = s["state_cache"][s["state_indices"]].float()
    S = S.mT if case["k_first"] else S
    if s["g"] is not None:
        S = s["g"].exp().expand(case["N"], -1)[..., None, None] * S
    delta = s["beta"].float()[..., None] * (v - (S @ k[..., None])[..., 0])
    S = S + delta[..., :, None] * k[..., None, :]
    out = (s["scale"] * (S @ q[..., None])[..., 0]).to(s["v"].dtype)
    s["state_cache"][s["state_indices"]] = (S.mT if case["k_first"] else S).to(s["state_cache"].dtype)
    return {"out": out, "state": s["state_cache"]}


def _norm(s):
    case = s["case"]
    kw = dict(kind=case["kind"], eps=EPS, weight_offset=case["offset"], interleaved=case["interleaved"])
    if own:
        import gated_delta_rule_pack_amd as kda
        rest = (s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["inv_freq"])
        if not case["back"]:
            q, k = kda.qk_norm(*rest, **kw)
            return {"q": q, "k": k}
        dq, dk, dqw, dkw = kda.qk_norm_backward(s["grad_q"], s["grad_k"], *rest, **kw)
        return {"q": dq, "k": dk, "q_weight": dqw, "k_weight": dkw}
    got = {}
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_weight"]
        share = 1 / case["D"] if case["kind"] == "rms" else 1.0
        inv = (share * x.square().sum(-1, keepdim=True) + EPS).rsqrt()
        scale = 1.0 if w is None else case["offset"] + w.float()
        if not case["back"]:
            got[n] = _plain_rotation(x * inv * scale, s, False).to(s[n].dtype)
            continue
        d = _plain_rotation(s["grad_" + n].float(), s, True)
        y = x * inv
        if w is None:
            got[n + "_weight"] = None
        else:
            got[n + "_weight"] = (d * y).sum((0, 1)).to(w.dtype)
        d = d * scale
        got[n] = (inv * (d - share * y * (d * y).sum(-1, keepdim=True))).to(s[n].dtype)
    return got


def _plain_rotation(x, s, inverse):
    """x [T, H, D] in 32 bits, its first 2 * len(inv_freq) channels rotated; angles in 64 bits."""
    if s["inv_freq"] is None:
        return x
    half = s["inv_freq"].numel()
    angle = (s["positions"].double()[:, None] * s["inv_freq"])[:, None]
    c, n = angle.cos().float(), (-angle if inverse else angle).sin().float()
    x, rest = x[..., : 2 * half], x[..., 2 * half :]
    interleaved = s["case"]["interleaved"]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    pair = (a * c - b * n, a * n + b * c)
    return torch.cat([torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1), rest], -1)


# ---------------------------------------------------------------------------- what a pass can not do without
def work(case):
    if case["op"] == "norm":
        es = 4 if case["dtype"] == "f32" else 2
        elems = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        small = (8 * case["T"] + 4 * case["rot"] if case["rot"] else 0) + 8 * case["D"] * (2 if case["back"] else 1)
        return {"bytes": (3 if case["back"] else 2) * elems * es + small, "flops": (12 if case["back"] else 6) * elems}
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
    tokens += T * H * (4 if case["beta"] == "f32" else 2)
    return {"bytes": tokens + planes * H * V * K * es, "flops": 6 * T * H * K * V}


# ---------------------------------------------------------------------------- 64 bits, from the definition
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    group = case["H"] // case["H_qk"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if case["normalize"]:
        q, k = (x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) for x in (q, k))
    begin, lens = list(range(q.shape[0])), [1] * q.shape[0]
    if case["op"] == "prompts":
        cu = s["cu_seqlens_cpu"].tolist()
        begin, lens = cu[:-1], [b - a for a, b in zip(cu, cu[1:])]
    lam = torch.ones(q.shape[0], case["H"], dtype=torch.float64, device=q.device)
    if s["g"] is not None:
        lam = lam * torch.exp(s["g"].double())
    beta = s["beta"].double()
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
        live.mul_(lam[row][:, :, None, None])
        off = v[row] - (live * kt[:, :, None, :]).sum(-1)
        live.addcmul_((beta[row][..., None] * off)[..., None], kt[:, :, None, :])
        out[row] = (live * qt[:, :, None, :]).sum(-1)
    back = torch.empty_like(S)
    back[where] = S
    back = back.transpose(-1, -2) if case["k_first"] else back
    if "initial_state" in s:
        return {"out": out * s["scale"], "state": back}
    pool = s["state_cache"].double()
    pool[slots] = back
    return {"out": out * s["scale"], "state": pool}


def _exact_norm(case, s):
    """The rotation as a product with complex numbers; the gradient by the product rule on numerator and length."""
    got = {}
    for n in ("q", "k"):
        x, w = s[n].double(), s[n + "_weight"]
        length = torch.sqrt((x * x).sum(-1, keepdim=True) / (case["D"] if case["kind"] == "rms" else 1) + EPS)
        w = None if w is None else case["offset"] + w.double()
        if not case["back"]:
            y = x / length
            got[n] = _turn(y if w is None else y * w, s, 1.0)
            continue
        d = _turn(s["grad_" + n].double(), s, -1.0)
        got[n + "_weight"] = None if w is None else torch.einsum("thd,thd->d", d, x / length)
        d = d if w is None else d * w
        slope = (d * x).sum(-1, keepdim=True) / (length ** 3 * (case["D"] if case["kind"] == "rms" else 1))
        got[n] = d / length - x * slope
    return got


def _turn(x, s, sign):
    if s["inv_freq"] is None:
        return x
    half, interleaved = s["inv_freq"].numel(), s["case"]["interleaved"]
    head, rest = x[..., : 2 * half], x[..., 2 * half :]
    pairs = head.unflatten(-1, (half, 2)) if interleaved else head.unflatten(-1, (2, half)).transpose(-1, -2)
    angle = sign * s["positions"].double()[:, None] * s["inv_freq"]
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None]
    pairs = torch.view_as_real(z)
    head = pairs.flatten(-2) if interleaved else pairs.transpose(-1, -2).flatten(-2)
    return torch.cat([head, rest], -1)
