"""What completes a diffusion-transformer block beside AdaLN, the rotations and the gated feed-forward, as measured cases:
linear attention with a decay for each head ("lin"), the join of a branch with the residual stream, with AdaLN's gate
and dropout from a counter-based generator ("residual"), and the way of tokens to the experts of a mixture and back
("experts"), each with its plain form in elementary torch operations and its definition in 64 bits.

A lin case: B samples of N tokens, H heads of d features; `pass` "fwd", "train" (forward and gradients) or "step" (one
token of each sample, N = 1, from state to state); `state`: the sequences continue an earlier state and hand theirs on;
"qkv": q, k and v are views of one fused projection's output.  A residual case: B samples of N tokens of D features,
dropout rate p, a gate vector for each sample or none.  An experts case: T tokens of D features, k choices of E experts
each, a share `lost` of them dropped (no expert)."""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lin(name, pas, B, N, H, d, dtype, state=False, qkv=False):
    return {"name": name, "op": "lin", "pass": pas, "B": B, "N": N, "H": H, "d": d, "dtype": dtype, "state": state,
            "qkv": qkv}


def _residual(name, pas, B, N, D, p, dtype, gate=True):
    return {"name": name, "op": "residual", "pass": pas, "B": B, "N": N, "D": D, "p": p, "dtype": dtype, "gate": gate}


def _experts(name, pas, T, k, E, D, dtype, lost=0.0):
    return {"name": name, "op": "experts", "pass": pas, "T": T, "k": k, "E": E, "D": D, "dtype": dtype, "lost": lost}


def listed():
    return [
        # one token of one stream, a step of generation: all latency
        _lin("lin_step_one", "step", 1, 1, 12, 128, "bf16"),
        # 64 streams generated together: the states' bytes are the work
        _lin("lin_step_batch", "step", 64, 1, 24, 128, "bf16"),
        # a prompt of 21 x 30 x 52 latent tokens, straight from the projection
        _lin("lin_video", "fwd", 1, 32760, 24, 128, "bf16", state=True, qkv=True),
        # a training step on 16 images of 30 x 52 latent tokens
        _lin("lin_images_train", "train", 16, 1560, 12, 128, "bf16", qkv=True),
        # odd sizes in f32, a chunk of a longer video trained through its state
        _lin("lin_ragged_f32", "train", 2, 1777, 10, 72, "f32", state=True),
        # a few conditioning tokens joined in sampling, no dropout
        _residual("residual_few", "fwd", 8, 1, 1536, 0.0, "bf16"),
        # odd sizes in f32
        _residual("residual_ragged_f32", "train", 3, 1111, 1156, 0.25, "f32"),
        # the large model's video, 21 x 45 x 80 latent tokens, forward and gradients
        _residual("residual_large_train", "train", 1, 75600, 5120, 0.1, "bf16"),
        # a few tokens of sampling to 2 of 16 experts
        _experts("experts_few", "fwd", 8, 2, 16, 1536, "bf16"),
        # ragged in every size, some choices dropped
        _experts("experts_ragged_f32", "train", 777, 3, 60, 1000, "f32", lost=0.1),
        # 16 images of 1560 tokens to 2 of 8 experts, a training step
        _experts("experts_images_train", "train", 24960, 2, 8, 1536, "bf16"),
        # a wide model's video, 4 of 64 experts
        _experts("experts_large_train", "train", 32760, 4, 64, 5120, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin", "lin", "residual", "experts"])
    while True:
        dtype = rng.choice(["bf16", "bf16", "f32"])
        e, unit = (2, 8) if dtype == "bf16" else (4, 4)
        if op == "lin":
            pas = rng.choice(["fwd", "train", "train", "step"])
            c = {"op": op, "pass": pas, "B": _log(rng, 1, 64), "N": 1 if pas == "step" else _log(rng, 1, 32760),
                 "H": rng.randint(1, 40), "d": unit * rng.randint(16 // unit, 128 // unit), "dtype": dtype,
                 "state": rng.random() < 0.5, "qkv": rng.random() < 0.5}
            if c["B"] * c["N"] * c["H"] * c["d"] * e <= 24960 * 12 * 128 * 2 and c["B"] * c["H"] <= 64 * 24:
                return c
        elif op == "residual":
            c = {"op": op, "pass": rng.choice(["fwd", "train"]), "B": _log(rng, 1, 64), "N": _log(rng, 1, 75600),
                 "D": unit * _log(rng, 64 // unit, 8192 // unit), "p": rng.choice([0.0, 0.05, 0.1, 0.5]),
                 "dtype": dtype, "gate": rng.random() < 0.8}
            if c["B"] * c["N"] * c["D"] * e <= 75600 * 5120 * 2:
                return c
        else:
            E = _log(rng, 2, 256)
            c = {"op": op, "pass": rng.choice(["fwd", "train"]), "T": _log(rng, 1, 131072),
                 "k": rng.randint(1, min(8, E)), "E": E, "D": unit * _log(rng, 64 // unit, 8192 // unit),
                 "dtype": dtype, "lost": rng.choice([0.0, 0.0, 0.2])}
            if c["T"] * c["k"] * c["D"] * e <= 32760 * 4 * 5120 * 2:
                return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "lin":
        B, N, H, d = (case[n] for n in ("B", "N", "H", "d"))
        n, states = B * N * H * d, 4 * B * H * d * d
        if case["pass"] == "step":
            return {"bytes": 2 * states + 4 * e * n, "flops": 6 * n * d}
        # chunks of min(N, d) tokens: within a chunk and through the state, which costs least
        c = min(N, d)
        fwd = n * (2 * c + 4 * d)
        held = states if case["state"] else 0
        if case["pass"] == "fwd":
            return {"bytes": 4 * e * n + 2 * held, "flops": fwd}
        # q, k, v and do in, dq, dk and dv out; states in, their gradients in and out
        return {"bytes": 11 * e * n + 5 * held, "flops": 3 * fwd}
    if case["op"] == "residual":
        B, N, D = case["B"], case["N"], case["D"]
        n, g = B * N * D, B * D if case["gate"] else 0
        if case["pass"] == "fwd":
            return {"bytes": 3 * e * n + e * g, "flops": 3 * n}
        bwd = (3 if case["gate"] else 2) * e * n + (e + 4) * g
        return {"bytes": 3 * e * n + e * g + bwd, "flops": 8 * n}
    T, k, D = case["T"], case["k"], case["D"]
    n = T * D
    choices = 8 * T * k + 4 * case["E"]
    fwd = 2 * e * n * (1 + k) + 4 * T * k
    if case["pass"] == "fwd":
        return {"bytes": choices + fwd, "flops": 2 * n * k}
    # dy and ys in, dys out; dxs in, dx out
    return {"bytes": choices + fwd + e * n * (1 + 2 * k) + e * n * (1 + k) + 8 * T * k, "flops": 6 * n * k}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    train = case["pass"] == "train"

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = {"case": case}
    if case["op"] == "lin":
        B, N, H, d = (case[n] for n in ("B", "N", "H", "d"))
        if case["pass"] == "step":
            s["q"], s["k"], s["v"] = normal(B, H, d), normal(B, H, d), normal(B, H, d)
            s["state"], s["next"] = normal(B, H, d, d, std=4.0, dtype=torch.float32), \
                torch.empty(B, H, d, d, device=dev)
        elif case["qkv"]:
            x = normal(B, N, 3 * H * d)
            s["q"], s["k"], s["v"] = (x[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
        else:
            s["q"], s["k"], s["v"] = normal(B, N, H, d), normal(B, N, H, d), normal(B, N, H, d)
        # heads that remember some 8 tokens up to some 4000, as decays are spread over heads
        span = 2.0 ** (3 + 9 * (torch.arange(H, device=dev) + torch.rand(H, generator=g, device=dev)) / H)
        s["log_decay"] = torch.log1p(-1 / span).float()
        if case["state"] and case["pass"] != "step":
            s["state"] = normal(B, H, d, d, std=4.0, dtype=torch.float32)
        if train:
            s["do"] = normal(B, N, H, d, std=1e-2)
            if case["state"]:
                s["dstate_out"] = normal(B, H, d, d, std=1e-2, dtype=torch.float32)
        return s
    if case["op"] == "residual":
        B, N, D = case["B"], case["N"], case["D"]
        s["x"], s["h"] = normal(B, N, D), normal(B, N, D)
        s["gate"] = normal(B, D, std=0.5) if case["gate"] else None
        # seed of the run and number of the call
        s["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=g, device=dev, dtype=torch.int64)
        if train:
            s["dy"] = normal(B, N, D, std=1e-2)
        return s
    T, k, E, D = (case[n] for n in ("T", "k", "E", "D"))
    # a router's choices, some experts liked more than others, and its weights
    scores = normal(T, E, dtype=torch.float32) + normal(E, dtype=torch.float32)
    top, expert = scores.topk(k, -1)
    if case["lost"]:
        lost = torch.rand(T, k, generator=g, device=dev) < case["lost"]
        expert = torch.where(lost, torch.full_like(expert, -1), expert)
    s["expert"], s["w"] = expert.to(torch.int32), torch.softmax(top, -1)
    s["x"], s["ys"] = normal(T, D), normal(T * k, D)
    # sorted rows that no choice fills are left as they are
    s["xs"] = torch.zeros(T * k, D, device=dev, dtype=dt)
    if train:
        s["dy"], s["dxs"] = normal(T, D, std=1e-2), normal(T * k, D, std=1e-2)
        s["dys"] = torch.zeros(T * k, D, device=dev, dtype=dt)
    return s


# ------------------------------------------------------------------ plain forms


def _chunked(q, k, v, g, c, state, C=64):
    """[B, N, H, d] in 32 bits; returns o and the state behind the last token."""
    B, N, H, d = q.shape
    n = -(-N // C)

    def chunks(x):
        out = x.new_zeros(B, H, n * C, d)
        out[:, :, :N] = x.transpose(1, 2)
        return out.view(B, H, n, C, d)

    q, k, v = chunks(q), chunks(k), chunks(v)
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    g = g[:, None]
    near = torch.where(i[:, None] >= i, torch.exp(g[..., None] * (i[:, None] - i).clamp(min=0)), 0.0)
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2).contiguous()) * near[:, None], v)
    last = N - (n - 1) * C
    kv = torch.matmul((k * torch.exp(g * (C - 1 - i))[:, None, :, None]).transpose(-1, -2).contiguous(), v)
    over = torch.exp(g * C)[..., None]
    s = torch.zeros_like(kv[:, :, 0]) if state is None else state
    before = []
    for j in range(n):
        before.append(s)
        if j < n - 1:
            s = s * over + kv[:, :, j]
    o = o + torch.matmul(q, torch.stack(before, 2)) * torch.exp(g * (i + 1))[:, None, :, None]
    # the last chunk ends where the tokens end
    tail = torch.exp(g * (last - 1 - i[:last]))[..., None]
    s = s * torch.exp(g * last)[..., None] + \
        torch.matmul((k[:, :, -1, :last] * tail).transpose(-1, -2).contiguous(), v[:, :, -1, :last])
    return (c * o).reshape(B, H, n * C, d)[:, :, :N].transpose(1, 2), s


def _lin_plain(s):
    case = s["case"]
    g, c = s["log_decay"], case["d"] ** -0.5
    q, k, v = (s[n].float() for n in "qkv")
    dt = s["q"].dtype
    if case["pass"] == "step":
        new = s["state"] * torch.exp(g)[:, None, None] + k[..., None] * v[..., None, :]
        return {"o": (c * (q[..., None] * new).sum(-2)).to(dt), "state": new}
    state = s.get("state")
    o, last = _chunked(q, k, v, g, c, state)
    out = {"o": o.to(dt)}
    if state is not None:
        out["state"] = last
    if case["pass"] == "train":
        do = s["do"].float()
        dlast = s.get("dstate_out")
        t = (lambda x: None if x is None else x.transpose(-1, -2).contiguous())
        # the gradients are the same operator with other parts; dk and dv from the last token to the first
        out["dq"] = _chunked(do, v, k, g, c, t(state))[0].to(dt)
        qr, kr, vr, dr = (x.flip(1) for x in (q, k, v, do))
        # the last token takes the state's gradient undecayed, where the operator would decay it once
        one = torch.exp(g)[:, None, None]
        back = None if dlast is None else dlast / (c * one)
        dv, ds = _chunked(kr, qr, dr, g, c, back)
        dk, _ = _chunked(vr, dr, qr, g, c, t(back))
        out["dk"], out["dv"] = dk.flip(1).to(dt), dv.flip(1).to(dt)
        if state is not None:
            out["dstate"] = c * one * ds
    return out


def _words(rng, rows, D):
    """Philox 4x32 in ten rounds: 8 x 16 random bits for each 8 features of a row, as int64 [rows, ceil(D / 8), 8].
    Products wrap around in 64 bits, which leaves their two words right."""
    m = 0xFFFFFFFF
    per = -(-D // 8)
    block = torch.arange(rows * per, device=rng.device, dtype=torch.int64)
    x = [block & m, (block >> 32) & m, (rng[1] & m).expand_as(block), ((rng[1] >> 32) & m).expand_as(block)]
    k0, k1 = rng[0] & m, (rng[0] >> 32) & m
    for r in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [((b >> 32) & m) ^ x[1] ^ k0, b & m, ((a >> 32) & m) ^ x[3] ^ k1, a & m]
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    halves = [h for w in x for h in (w & 0xFFFF, w >> 16)]
    return torch.stack(halves, -1).view(rows, per, 8)


def _residual_plain(s):
    case = s["case"]
    B, N, D, p = case["B"], case["N"], case["D"], case["p"]
    dt = s["h"].dtype
    h = s["h"].float()
    if p > 0:
        limit = int(math.floor((1 - p) * 65536 + 0.5))
        keep = (_words(s["rng"], B * N, D) < limit).view(B, N, -1)[..., :D]
        h = torch.where(keep, h * (65536 / limit), 0.0)
    gate = None if s["gate"] is None else s["gate"].float()[:, None]
    out = {"y": (s["x"].float() + (h if gate is None else gate * h)).to(dt)}
    if case["pass"] == "train":
        dy = s["dy"].float()
        if gate is not None:
            out["dgate"] = (dy * h).sum(1)
            dh = dy * gate
        else:
            dh = dy
        out["dh"] = (torch.where(keep, dh * (65536 / limit), 0.0) if p > 0 else dh).to(dt)
    return out


def _experts_plain(s):
    case = s["case"]
    T, k, E, D = (case[n] for n in ("T", "k", "E", "D"))
    flat = s["expert"].flatten().long()
    there = (flat >= 0) & (flat < E)
    order = torch.argsort(torch.where(there, flat, torch.full_like(flat, E)), stable=True)
    rows = torch.arange(T * k, device=flat.device)
    slot = torch.empty_like(flat)
    slot[order] = rows
    slot = torch.where(there, slot, torch.full_like(slot, -1))
    count = torch.zeros(E + 1, device=flat.device, dtype=torch.int64)
    count[1:] = (flat[there][:, None] == torch.arange(E, device=flat.device)).sum(0) if T * k * E < 1 << 24 else \
        torch.zeros(E, device=flat.device, dtype=torch.int64).index_add_(0, flat[there], torch.ones_like(flat[there]))
    out = {"offsets": count.cumsum(0).to(torch.int32), "slot": slot.view(T, k).to(torch.int32)}
    full = rows < out["offsets"][-1]
    dt = s["x"].dtype
    x, w = s["x"].float(), s["w"]
    out["xs"] = torch.where(full[:, None], x[order // k], s["xs"].float()).to(dt)
    at, on = slot.clamp(min=0).view(T, k), there.view(T, k, 1)
    ys = s["ys"].float()
    out["y"] = sum(torch.where(on[:, j], w[:, j, None] * ys[at[:, j]], 0.0) for j in range(k)).to(dt)
    if case["pass"] == "train":
        dy, dxs = s["dy"].float(), s["dxs"].float()
        out["dys"] = torch.where(full[:, None], w.flatten()[order, None] * dy[order // k], s["dys"].float()).to(dt)
        out["dw"] = torch.stack([torch.where(on[:, j, 0], (dy * ys[at[:, j]]).sum(-1), 0.0) for j in range(k)], -1)
        out["dx"] = sum(torch.where(on[:, j], dxs[at[:, j]], 0.0) for j in range(k)).to(dt)
    return out


_PLAIN = {"lin": _lin_plain, "residual": _residual_plain, "experts": _experts_plain}


# ------------------------------------------------------- the framework's calls


def _kernels(s):
    import adaln_fwd_amd as A
    case = s["case"]
    out = {}
    train = case["pass"] == "train"
    if case["op"] == "lin":
        if case["pass"] == "step":
            out["o"], out["state"] = A.lin_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                                                     state_out=s["next"])
            return out
        state = s.get("state")
        o, last, saved = A.lin_attn_fwd(s["q"], s["k"], s["v"], s["log_decay"], state=state,
                                        final=state is not None, save=train)
        out["o"] = o
        if state is not None:
            out["state"] = last
        if train:
            out["dq"], out["dk"], out["dv"], dstate = A.lin_attn_bwd(
                s["do"], s["q"], s["k"], s["v"], s["log_decay"], state=state, saved=saved,
                dstate_out=s.get("dstate_out"))
            if state is not None:
                out["dstate"] = dstate
        return out
    if case["op"] == "residual":
        out["y"] = A.residual_fwd(s["x"], s["h"], s["gate"], p=case["p"], rng=s["rng"])
        if train:
            out["dh"], dgate = A.residual_bwd(s["dy"], s["h"], s["gate"], p=case["p"], rng=s["rng"])
            if dgate is not None:
                out["dgate"] = dgate
        return out
    out["offsets"], out["slot"] = A.experts_plan(s["expert"], case["E"])
    out["xs"] = A.experts_sort_fwd(s["x"], out["slot"], xs=s["xs"])
    out["y"] = A.experts_join_fwd(s["ys"], out["slot"], s["w"])
    if train:
        out["dys"], out["dw"] = A.experts_join_bwd(s["dy"], s["ys"], out["slot"], s["w"], dys=s["dys"])
        out["dx"] = A.experts_sort_bwd(s["dxs"], out["slot"])
    return out


def run(state):
    return _kernels(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits


def _exact_lin(case, s):
    B, N, H, d = (case[n] for n in ("B", "N", "H", "d"))
    c = 1 / math.sqrt(d)
    lam = s["log_decay"].double()
    if case["pass"] == "step":
        q, k, v = (s[n].double() for n in "qkv")
        new = torch.einsum("bhij,h->bhij", s["state"].double(), lam.exp()) + torch.einsum("bhi,bhj->bhij", k, v)
        return {"o": c * torch.einsum("bhi,bhij->bhj", q, new), "state": new}
    train = case["pass"] == "train"
    names = ["o", "dq", "dk", "dv"] if train else ["o"]
    out = {n: torch.zeros(B, N, H, d, dtype=torch.float64, device=lam.device) for n in names}
    S0, SN = s.get("state"), s.get("dstate_out")
    if S0 is not None:
        out["state"] = torch.zeros(B, H, d, d, dtype=torch.float64, device=lam.device)
        if train:
            out["dstate"] = torch.zeros_like(out["state"])
    t = torch.arange(N, device=lam.device, dtype=torch.float64)
    step = max(1, (1 << 27) // N)
    for b in range(B):
        for h in range(H):
            q, k, v = (s[n][b, :, h].double() for n in "qkv")
            do = s["do"][b, :, h].double() if train else None
            # every pair of tokens, rows of queries at a time
            for r in range(0, N, step):
                e = min(N, r + step)
                D = (t[r:e, None] - t[:e]) * lam[h]
                D = torch.where(t[:e] <= t[r:e, None], D.exp(), 0.0) * c
                P = (q[r:e] @ k[:e].T) * D
                out["o"][b, r:e, h] = P @ v[:e]
                if train:
                    dP = (do[r:e] @ v[:e].T) * D
                    out["dq"][b, r:e, h] = dP @ k[:e]
                    out["dk"][b, :e, h] += dP.T @ q[r:e]
                    out["dv"][b, :e, h] += P.T @ do[r:e]
            if S0 is not None:
                first, rest = torch.exp(lam[h] * (t + 1))[:, None], torch.exp(lam[h] * (N - 1 - t))[:, None]
                S = S0[b, h].double()
                all_ = torch.exp(lam[h] * N)
                out["o"][b, :, h] += c * first * (q @ S)
                out["state"][b, h] = all_ * S + (k * rest).T @ v
                if train:
                    dS = SN[b, h].double()
                    out["dq"][b, :, h] += c * first * (do @ S.T)
                    out["dk"][b, :, h] += rest * (v @ dS.T)
                    out["dv"][b, :, h] += rest * (k @ dS)
                    out["dstate"][b, h] = all_ * dS + c * (q * first).T @ do
    return out


def _exact_bits(rng, rows, D):
    """The generator from its definition, words as pairs of 16-bit limbs so that no product passes 2^53."""
    per = -(-D // 8)
    seed, call = (int(v) % 2 ** 64 for v in rng.cpu())
    block = torch.arange(rows * per, device=rng.device)

    def mul(word, const):
        lo, hi = word % 65536, word // 65536
        c0, c1 = const % 65536, const // 65536
        mid = lo * c1 + (lo * c0) // 65536
        mid2 = hi * c0 + mid % 65536
        return hi * c1 + mid // 65536 + mid2 // 65536, mid2 % 65536 * 65536 + (lo * c0) % 65536

    x = [block % 2 ** 32, block // 2 ** 32, torch.full_like(block, call % 2 ** 32),
         torch.full_like(block, call // 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        h0, l0 = mul(x[0], 0xD2511F53)
        h1, l1 = mul(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = torch.empty(rows * per, 8, device=rng.device, dtype=torch.int32)
    for i, w in enumerate(x):
        bits[:, 2 * i], bits[:, 2 * i + 1] = (w % 65536).int(), (w // 65536).int()
    return bits.view(rows, per * 8)[:, :D]


def _exact_residual(case, s):
    B, N, D = case["B"], case["N"], case["D"]
    limit = round((1 - case["p"]) * 65536)
    out = {"y": torch.empty(B, N, D, dtype=torch.float64, device=s["h"].device)}
    factor = torch.ones((), dtype=torch.float64, device=s["h"].device)
    if case["p"] > 0:
        factor = ((_exact_bits(s["rng"], B * N, D) < limit).to(torch.float64) * 65536 / limit).view(B, N, D)
    gate = torch.ones(B, D, dtype=torch.float64, device=s["h"].device) if s["gate"] is None else s["gate"].double()
    h = s["h"].double().mul_(factor)
    out["y"] = torch.addcmul(s["x"].double(), h, gate[:, None])
    if case["pass"] == "train":
        dy = s["dy"].double()
        if s["gate"] is not None:
            out["dgate"] = h.mul_(dy).sum(1)
        out["dh"] = dy.mul_(factor).mul_(gate[:, None])
    return out


def _exact_experts(case, s):
    T, k, E = case["T"], case["k"], case["E"]
    flat = s["expert"].flatten().tolist()
    lists = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(i)
    order = [i for part in lists for i in part]
    slots = [-1] * (T * k)
    for r, i in enumerate(order):
        slots[i] = r
    offsets = [0]
    for part in lists:
        offsets.append(offsets[-1] + len(part))
    dev = s["x"].device
    order = torch.tensor(order, device=dev, dtype=torch.int64)
    n = len(order)
    out = {"offsets": torch.tensor(offsets, device=dev, dtype=torch.int32),
           "slot": torch.tensor(slots, device=dev, dtype=torch.int32).view(T, k)}
    token, w = order // k, s["w"].flatten().double()[order]
    out["xs"] = s["xs"].double()
    out["xs"][:n] = s["x"].double()[token]
    # each token's sum, sorted rows one choice of the k at a time
    out["y"] = torch.zeros(s["x"].shape, dtype=torch.float64, device=dev)
    train = case["pass"] == "train"
    if train:
        out["dys"] = s["dys"].double()
        out["dw"] = torch.zeros(T * k, dtype=torch.float64, device=dev)
        out["dx"] = torch.zeros_like(out["y"])
    for j in range(k):
        r = torch.nonzero(order % k == j).flatten()
        t = token[r]
        out["y"][t] += s["ys"][r].double().mul_(w[r, None])
        if train:
            dy = s["dy"][t].double()
            out["dw"][order[r]] = torch.linalg.vecdot(dy, s["ys"][r].double())
            out["dys"][r] = dy.mul_(w[r, None])
            out["dx"][t] += s["dxs"][r].double()
    if train:
        out["dw"] = out["dw"].view(T, k)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"lin": _exact_lin, "residual": _exact_residual, "experts": _exact_experts}[case["op"]](case, s)
