"""The operators of a diffusion-transformer block run together as a training
step runs them, forward and backward: AdaLN, the query/key norms with the
rotation inside the projection's output, AdaLN again, the gated feed-forward;
torch's products stand for the projections around them.  Compared with the
same block in float64 through autograd."""

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu

B, N, H, HD, F = 2, 210, 4, 32, 328          # 2 x (5 x 6 x 7) tokens
D = H * HD
EPS = 1e-6


def _data():
    g = torch.Generator().manual_seed(11)

    def n(*s, std=1.0):
        return torch.randn(*s, generator=g) * std

    t = dict(x=n(B, N, D), s1=n(B, D, std=0.1), h1=n(B, D, std=0.1),
             s2=n(B, D, std=0.1), h2=n(B, D, std=0.1),
             wqkv=n(3 * D, D, std=D ** -0.5), wq=1 + n(HD, std=0.1),
             wk=1 + n(HD, std=0.1), wg=n(F, D, std=D ** -0.5),
             wu=n(F, D, std=D ** -0.5), wd=n(D, F, std=F ** -0.5),
             dq=n(B, N, H, HD), dk=n(B, N, H, HD), dy=n(B, N, D))
    t = {k: v.to(torch.bfloat16) for k, v in t.items()}
    i = torch.arange(N)
    pos = torch.stack([i // 42, i // 7 % 6, i % 7], -1).to(torch.int32)
    return t, pos, A.rope_freqs((6, 5, 5))


def _ln(x, s, h):
    m = x.mean(-1, keepdim=True)
    v = ((x - m) ** 2).mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(v + EPS) * (1 + s[:, None]) + h[:, None]


def _head(x, w, ang):
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    u, v = x[..., 0::2], x[..., 1::2]
    return torch.stack([u * c - v * s, u * s + v * c], -1).flatten(-2)


def _reference(t, pos, freqs):
    p = {k: v.double().requires_grad_(not k.startswith("d"))
         for k, v in t.items()}
    ang = pos.double() @ torch.from_numpy(freqs)
    qkv = _ln(p["x"], p["s1"], p["h1"]) @ p["wqkv"].t()
    q = _head(qkv[..., :D].unflatten(-1, (H, HD)), p["wq"], ang)
    k = _head(qkv[..., D:2 * D].unflatten(-1, (H, HD)), p["wk"], ang)
    z = _ln(p["x"], p["s2"], p["h2"])
    g = z @ p["wg"].t()
    y = (g / (1 + torch.exp(-g)) * (z @ p["wu"].t())) @ p["wd"].t()
    loss = (q * p["dq"]).sum() + (k * p["dk"]).sum() + (y * p["dy"]).sum()
    names = [n for n in p if not n.startswith("d")]
    grads = torch.autograd.grad(loss, [p[n] for n in names])
    return dict(q=q, k=k, y=y, **{"d_" + n: g for n, g in zip(names, grads)})


def _step(t, pos, freqs):
    """One forward and backward with the framework's operators."""
    z1, m1, r1 = A.fwd(t["x"], t["s1"], t["h1"])
    qkv = z1 @ t["wqkv"].t()
    q, k = (qkv[..., i * D:(i + 1) * D].unflatten(-1, (H, HD))
            for i in range(2))
    qo, ko = A.qk_norm_rope_fwd(q, k, t["wq"], t["wk"], pos, freqs, eps=EPS)
    z2, m2, r2 = A.fwd(t["x"], t["s2"], t["h2"])
    h, saved = A.glu_fwd(z2, t["wg"], t["wu"], save=True)
    y = h @ t["wd"].t()

    dh = t["dy"] @ t["wd"]
    dwd = t["dy"].flatten(0, 1).t() @ h.flatten(0, 1)
    dz2, dwg, dwu = A.glu_bwd(dh, z2, t["wg"], t["wu"], saved)
    dx2, ds2, dh2 = A.bwd(dz2, t["x"], t["s2"], m2, r2)
    # q and k's gradients land inside the projection's
    dqkv = torch.zeros_like(qkv)
    dq, dk = (dqkv[..., i * D:(i + 1) * D].unflatten(-1, (H, HD))
              for i in range(2))
    _, _, dwq, dwk = A.qk_norm_rope_bwd(t["dq"], t["dk"], q, k, t["wq"],
                                        t["wk"], pos, freqs, eps=EPS, dq=dq,
                                        dk=dk)
    dz1 = dqkv @ t["wqkv"]
    dwqkv = dqkv.flatten(0, 1).t() @ z1.flatten(0, 1)
    dx1, ds1, dh1 = A.bwd(dz1, t["x"], t["s1"], m1, r1)
    return dict(q=qo, k=ko, y=y, d_x=dx1.float() + dx2.float(), d_s1=ds1,
                d_h1=dh1, d_s2=ds2, d_h2=dh2, d_wqkv=dwqkv, d_wq=dwq,
                d_wk=dwk, d_wg=dwg, d_wu=dwu, d_wd=dwd)


def test_block_forward_and_backward():
    t, pos, freqs = _data()
    print("[block] forward and backward", flush=True)
    ref = _reference(t, pos, freqs)
    got = _step({k: v.cuda() for k, v in t.items()}, pos.cuda(), freqs)
    assert set(got) == set(ref)
    # Each path crosses at most eight roundings to bfloat16 (norm, projection,
    # rotation, its gradient, hidden, down, gradients between them), each at
    # most 2^-8 of a value and independent of the others: the 2-norm of an
    # output is off by at most sqrt(8) * 2^-8, and by twice that where a
    # norm's Jacobian amplifies (its gradient subtracts two projections).
    for n, r in ref.items():
        e = (got[n].double().cpu() - r).norm() / r.norm()
        print(f"[block]   {n}: {float(e):.2e}", flush=True)
        assert e < 2 * 8 ** 0.5 * 2 ** -8, n


def test_block_in_a_graph():
    t, pos, freqs = _data()
    print("[block] captured and replayed", flush=True)
    t = {k: v.cuda() for k, v in t.items()}
    pos = pos.cuda()
    want = {k: v.clone() for k, v in _step(t, pos, freqs).items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = _step(t, pos, freqs)
    keep = t["x"].clone()
    for i in range(3):
        t["x"].copy_(keep if i != 1 else keep * 0.5)
        eager = want if i != 1 else _step(t, pos, freqs)
        g.replay()
        torch.cuda.synchronize()
        for n in ("q", "k", "d_s1", "d_h1", "d_wq", "d_wk", "d_wg", "d_wu",
                  "d_s2", "d_h2"):
            assert torch.equal(outs[n], eager[n]), (i, n)
