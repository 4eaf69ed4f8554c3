"""A block with linear attention and experts run as a training step runs it,
forward and backward: AdaLN, the projections, the query/key norms with the
rotation and the linear attention inside the projection's output, the gated
join with dropout; AdaLN, the experts' plan and sort, each expert's gated
feed-forward, the join by weight, the gated join again.  torch's products stand
for the projections.  Compared with the same block in float64 through autograd;
and the block as serving runs it, the last tokens one at a time."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_lin_attn as RL
from tests import ref_residual as RR

pytestmark = pytest.mark.gpu

B, N, H, HD, F, E, K = 2, 210, 4, 32, 168, 5, 2      # 2 x (5 x 6 x 7) tokens
D, T = H * HD, B * N
EPS, P = 1e-6, 0.25
RNG = (1234567, 40)                                  # the second join: 41
LEAVES = ("x", "s1", "h1", "g1", "s2", "h2", "g2", "wqkv", "wq", "wk", "wo",
          "w", "wg", "wu", "wd")


def _data():
    g = torch.Generator().manual_seed(23)

    def n(*s, std=1.0):
        return torch.randn(*s, generator=g) * std

    t = dict(x=n(B, N, D), s1=n(B, D, std=0.1), h1=n(B, D, std=0.1),
             g1=1 + n(B, D, std=0.1), s2=n(B, D, std=0.1),
             h2=n(B, D, std=0.1), g2=1 + n(B, D, std=0.1),
             wqkv=n(3 * D, D, std=D ** -0.5), wq=1 + n(HD, std=0.1),
             wk=1 + n(HD, std=0.1), wo=n(D, D, std=D ** -0.5),
             wg=n(E, F, D, std=D ** -0.5), wu=n(E, F, D, std=D ** -0.5),
             wd=n(E, D, F, std=F ** -0.5), dy=n(B, N, D))
    t = {k: v.to(torch.bfloat16) for k, v in t.items()}
    t["w"] = torch.softmax(n(T, K), -1)
    expert = torch.randint(0, E, (T, K), generator=g)
    expert[expert[:, 0] == expert[:, 1], 1] = E      # dropped
    t["expert"] = expert
    t["decay"] = torch.log1p(-(2.0 ** -torch.arange(2., 2. + H)))
    i = torch.arange(N)
    t["pos"] = torch.stack([i // 42, i // 7 % 6, i % 7], -1).to(torch.int32)
    return t


FREQS = A.rope_freqs((6, 5, 5))


def _ln(x, s, h):
    m = x.mean(-1, keepdim=True)
    v = ((x - m) ** 2).mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(v + EPS) * (1 + s[:, None]) + h[:, None]


def _head(x, w, ang):
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)


def _reference(t, rng=RNG):
    p = {k: t[k].double().requires_grad_() for k in LEAVES}
    ang = t["pos"].double() @ torch.from_numpy(FREQS)

    def drop(call):
        keep, s = RR.keep_mask(T, D, P, (rng[0], call))
        return torch.as_tensor(keep).double().view(B, N, D) * s

    qkv = _ln(p["x"], p["s1"], p["h1"]) @ p["wqkv"].t()
    q, k, v = (qkv[..., i * D:(i + 1) * D].unflatten(-1, (H, HD))
               for i in range(3))
    q, k = _head(q, p["wq"], ang), _head(k, p["wk"], ang)
    # o_t = sum over s <= t of l^(t - s) (q_t . k_s) v_s / sqrt(d)
    gap = torch.arange(N)[:, None] - torch.arange(N)
    power = torch.where(gap >= 0, torch.exp(t["decay"].double()[:, None, None]
                                            * gap.clamp(min=0)), 0.0)
    a = torch.einsum("bthd,bshd->bhts", q, k) * power * HD ** -0.5
    o = torch.einsum("bhts,bshd->bthd", a, v)
    x2 = p["x"] + p["g1"][:, None] * drop(rng[1]) * (o.flatten(2) @
                                                     p["wo"].t())
    z = _ln(x2, p["s2"], p["h2"]).view(T, D)
    y = torch.zeros_like(z)
    for j in range(K):
        for e in range(E):
            rows = torch.nonzero(t["expert"][:, j] == e).flatten()
            g = z[rows] @ p["wg"][e].t()
            out = (g * torch.sigmoid(g) * (z[rows] @ p["wu"][e].t())) @ \
                p["wd"][e].t()
            y = y.index_add(0, rows, p["w"][rows, j, None] * out)
    y = x2 + p["g2"][:, None] * drop(rng[1] + 1) * y.view(B, N, D)
    grads = torch.autograd.grad((y * t["dy"].double()).sum(),
                                [p[n] for n in LEAVES])
    return dict(o=o, y=y, **{"d_" + n: g for n, g in zip(LEAVES, grads)})


def _step(t, rng, at):
    """One forward and backward; at: the experts' offsets on the host."""
    x = t["x"]
    z1, m1, r1 = A.fwd(x, t["s1"], t["h1"])
    qkv = z1 @ t["wqkv"].t()
    q, k, v = (qkv[..., i * D:(i + 1) * D].unflatten(-1, (H, HD))
               for i in range(3))
    qo, ko = A.qk_norm_rope_fwd(q, k, t["wq"], t["wk"], t["pos"], FREQS,
                                eps=EPS)
    o, _, states = A.lin_attn_fwd(qo, ko, v, t["decay"], save=True)
    a = o.flatten(2) @ t["wo"].t()
    rng2 = rng.clone()
    rng2[1] += 1
    x2 = A.residual_fwd(x, a, t["g1"], p=P, rng=rng)
    z2, m2, r2 = A.fwd(x2, t["s2"], t["h2"])
    offsets, slot = A.experts_plan(t["expert"], E)
    zs = A.experts_sort_fwd(z2.view(T, D), slot)
    ys = torch.zeros_like(zs)
    hs, saves = [], []
    for e in range(E):
        h, s = A.glu_fwd(zs[at[e]:at[e + 1]], t["wg"][e], t["wu"][e],
                         save=True)
        hs.append(h), saves.append(s)
        torch.mm(h, t["wd"][e].t(), out=ys[at[e]:at[e + 1]])
    f = A.experts_join_fwd(ys, slot, t["w"])
    y = A.residual_fwd(x2, f.view(B, N, D), t["g2"], p=P, rng=rng2)

    df, dg2 = A.residual_bwd(t["dy"], f.view(B, N, D), t["g2"], p=P, rng=rng2)
    dys, dw = A.experts_join_bwd(df.view(T, D), ys, slot, t["w"])
    dzs = torch.zeros_like(zs)
    dwg, dwu, dwd = [], [], []
    for e in range(E):
        d = dys[at[e]:at[e + 1]]
        dz, g, u = A.glu_bwd(d @ t["wd"][e], zs[at[e]:at[e + 1]], t["wg"][e],
                             t["wu"][e], saves[e])
        dzs[at[e]:at[e + 1]].copy_(dz)
        dwg.append(g), dwu.append(u), dwd.append(d.t() @ hs[e])
    dz2 = A.experts_sort_bwd(dzs, slot).view(B, N, D)
    dx2, ds2, dh2 = A.bwd(dz2, x2, t["s2"], m2, r2)
    dx2 = A.residual_fwd(t["dy"], dx2)               # the two paths' sum
    da, dg1 = A.residual_bwd(dx2, a, t["g1"], p=P, rng=rng)
    do = (da @ t["wo"]).unflatten(-1, (H, HD))
    dwo = da.flatten(0, 1).t() @ o.flatten(2).flatten(0, 1)
    dqkv = torch.zeros_like(qkv)
    dq, dk, dv = (dqkv[..., i * D:(i + 1) * D].unflatten(-1, (H, HD))
                  for i in range(3))
    dqo, dko, _, _ = A.lin_attn_bwd(do, qo, ko, v, t["decay"], saved=states,
                                    dv=dv)
    _, _, dwq, dwk = A.qk_norm_rope_bwd(dqo, dko, q, k, t["wq"], t["wk"],
                                        t["pos"], FREQS, eps=EPS, dq=dq,
                                        dk=dk)
    dz1 = dqkv @ t["wqkv"]
    dwqkv = dqkv.flatten(0, 1).t() @ z1.flatten(0, 1)
    dx1, ds1, dh1 = A.bwd(dz1, x, t["s1"], m1, r1)
    return dict(o=o, y=y, d_x=A.residual_fwd(dx2, dx1), d_s1=ds1, d_h1=dh1,
                d_g1=dg1, d_s2=ds2, d_h2=dh2, d_g2=dg2, d_wqkv=dwqkv,
                d_wq=dwq, d_wk=dwk, d_wo=dwo, d_w=dw, d_wg=torch.stack(dwg),
                d_wu=torch.stack(dwu), d_wd=torch.stack(dwd)), offsets


def _offsets(t):
    n = torch.bincount(t["expert"].flatten(), minlength=E + 1)[:E]
    return [0] + n.cumsum(0).tolist()


def test_block_forward_and_backward():
    t = _data()
    at = _offsets(t)
    ref = _reference(t)
    print("[linear block] forward and backward", flush=True)
    got, offsets = _step({k: v.cuda() for k, v in t.items()},
                         torch.tensor(RNG, device="cuda"), at)
    assert offsets.tolist() == at and set(got) == set(ref)
    # The longest path, x's gradient, crosses twenty-six roundings to bfloat16
    # (thirteen of values: norm, projection, rotation, attention, projection,
    # join, norm, two of the feed-forward, its hidden, down, join, join; and
    # as many of gradients), each at most 2^-8 of a value and independent of
    # the others: the 2-norm of an output is off by at most sqrt(26) * 2^-8,
    # and by twice that where a norm's Jacobian amplifies.
    for n, r in ref.items():
        e = (got[n].double().cpu() - r.detach()).norm() / r.detach().norm()
        print(f"[linear block]   {n}: {float(e):.2e}", flush=True)
        assert e < 2 * 26 ** 0.5 * 2 ** -8, n


def test_block_in_a_graph():
    t = _data()
    at = _offsets(t)
    t = {k: v.cuda() for k, v in t.items()}
    rng = torch.tensor(RNG, device="cuda")
    print("[linear block] captured and replayed", flush=True)

    def eager():
        return {k: v.clone() for k, v in _step(t, rng, at)[0].items()}

    eager()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs, offsets = _step(t, rng, at)
        rng[1] += 2                                  # the next step's numbers
    keep, seen = t["x"].clone(), []
    for i in range(4):
        t["x"].copy_(keep if i != 1 else keep * 0.5)
        call = int(rng[1])
        assert call == RNG[1] + 2 * i
        want = eager()
        g.replay()
        torch.cuda.synchronize()
        for n in ("o", "y", "d_x", "d_s1", "d_h1", "d_g1", "d_s2", "d_h2",
                  "d_g2", "d_wq", "d_wk", "d_w", "d_wg", "d_wu"):
            assert torch.equal(outs[n], want[n]), (i, n)
        assert offsets.tolist() == at
        seen.append(outs["y"].clone())
    assert not torch.equal(seen[0], seen[2])         # other elements dropped


def test_block_served_token_by_token():
    """The attention's half on a prefix, its state, then single tokens."""
    t = _data()
    prefix, more = 203, N - 203
    d = {k: v.cuda() for k, v in t.items()}
    print("[linear block] a prefix and single tokens", flush=True)

    def front(x, at):
        n = x.shape[1]
        z, _, _ = A.fwd(x, d["s1"], d["h1"])
        qkv = z @ d["wqkv"].t()
        q, k, v = (qkv[..., i * D:(i + 1) * D].unflatten(-1, (H, HD))
                   for i in range(3))
        q, k = A.qk_norm_rope_fwd(q, k, d["wq"], d["wk"],
                                  d["pos"][at:at + n].contiguous(), FREQS,
                                  eps=EPS)
        return q, k, v

    q, k, v = front(d["x"][:, :prefix].contiguous(), 0)
    ins = [[y.cpu()] for y in (q, k, v)]
    o, state, _ = A.lin_attn_fwd(q, k, v, d["decay"], final=True)
    outs = [o]
    for i in range(more):
        x = d["x"][:, prefix + i:prefix + i + 1].contiguous()
        q, k, v = front(x, prefix + i)
        for seen, y in zip(ins, (q, k, v)):
            seen.append(y.cpu())
        o, same = A.lin_attn_step(q[:, 0], k[:, 0], v[:, 0], d["decay"], state)
        assert same is state
        outs.append(o[:, None])
        y = A.residual_fwd(x, o.flatten(1)[:, None].contiguous(), d["g1"])
        assert torch.isfinite(y).all()
    got = torch.cat(outs, 1).double().cpu()
    q, k, v = (torch.cat(s, 1) for s in ins)
    for b in range(B):
        args = (q[b], k[b], v[b], t["decay"], HD ** -0.5)
        want, end = RL.forward(*args)
        big, most = RL.forward(*args, sums=True)
        # of the terms' absolute values: the two parts of the scores and the
        # states, and of the products with both, 2^-16 each, and the float32
        # sums, at most N / 8 + 4 d + 64 roundings; of the output half a step
        rel = (N / 8 + 4 * HD + 64) * 2.0 ** -24
        err = (got[b] - want).abs()
        assert (err <= 2.0 ** -8 * (want.abs() + rel * big)
                + (rel + 3 * 2.0 ** -16) * big).all(), b
        # the states are sums of three parts
        err = (state[b].double().cpu() - end).abs()
        assert (err <= rel * most).all(), b
