"""Plain 64-bit forms of sink attention and of the shared-prefix decode step,
written row by row from their definitions (tests only), and the inputs of the
tests.  The forward without sinks is pinned to the oracle, the gradients to central
differences, in test_sink_ref.py."""
import math

import torch

D, W, EPS = 128, 128, 1e-6


def norm_rope(x, w, pos, R, base, eps=EPS):
    """RoPE_pos(x / rms(x) * w); x [..., H, 128], pos of x's leading axes."""
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w
    h = R // 2
    if h == 0:
        return y
    f = base ** (-2.0 * torch.arange(h, dtype=torch.float64) / R)
    a = pos.double()[..., None, None] * f
    c, s = a.cos(), a.sin()
    u, v = y[..., :h], y[..., h:R]
    return torch.cat([u * c - v * s, v * c + u * s, y[..., R:]], -1)


def visible(i, n_sink, T):
    """Keys that query i attends, in order."""
    return [j for j in range(T) if j <= i and (i - j < W or j < n_sink)]


def sink_forward(q, k, v, g, wq, wk, n_sink, R, base, scale=0.0):
    """o and lse of the whole batch, fp64 (differentiable)."""
    B, T, Hq, _ = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    scale = scale or 1.0 / math.sqrt(D)
    pos = torch.arange(T).expand(B, T)
    qq, kk = norm_rope(q, wq, pos, R, base), norm_rope(k, wk, pos, R, base)
    o, lse = [], []
    for i in range(T):
        js = visible(i, n_sink, T)
        x = torch.einsum("bhgd,bjhd->bhgj", qq[:, i].reshape(B, Hkv, G, D), kk[:, js]) * scale
        lse.append(torch.logsumexp(x, -1).reshape(B, Hq))
        a = torch.einsum("bhgj,bjhd->bhgd", torch.softmax(x, -1), v[:, js]).reshape(B, Hq, D)
        o.append(a * torch.sigmoid(g[:, i]))
    return torch.stack(o, 1), torch.stack(lse, 2)


def sink_gradients(x, dO, n_sink, R, base, scale=0.0):
    """Gradients of sum(o dO) for x = (q, k, v, g, wq, wk) in fp64."""
    x = [t.double().clone().requires_grad_() for t in x]
    o, _ = sink_forward(*x, n_sink, R, base, scale)
    return torch.autograd.grad((o * dO.double()).sum(), x)


def context_attention(q, k, v, scale=0.0):
    """One sequence's token: q [Hq, D] against k, v [Hkv, n, D] (all visible), fp64."""
    Hkv = k.shape[0]
    x = torch.einsum("hgd,hnd->hgn", q.reshape(Hkv, -1, D), k) * (scale or 1.0 / math.sqrt(D))
    return torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v).reshape(q.shape)


def draw(B, T, Hq, Hkv, seed, g_std=1.0, grad=False):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(s, generator=gen) * std).to(torch.bfloat16)
    x = dict(q=n(B, T, Hq, D), k=n(B, T, Hkv, D), v=n(B, T, Hkv, D), g=n(B, T, Hq, D, std=g_std),
             wq=1 + 0.1 * torch.randn(D, generator=gen), wk=1 + 0.1 * torch.randn(D, generator=gen))
    if grad:
        x["dO"] = n(B, T, Hq, D)
    return x


NAMES = ("q", "k", "v", "g", "wq", "wk")


def args(x, dev=None, dtype=None):
    t = [x[n] for n in NAMES]
    if dev is not None:
        t = [y.to(dev) for y in t]
    return [y.to(dtype) for y in t] if dtype is not None else t


def rel(got, ref):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    return float((got - ref).norm() / ref.norm().clamp_min(1e-300))


def neighbours(got, want):
    """Where a bf16 cache holds the same bits as the 64-bit form's, or an entry that fp32
    arithmetic may round otherwise: k' = u c - v s of |u|, |v| <= 12 max|w| < 16.9 with six
    fp32 roundings, 6 x 2^-24 x 2 x 16.9 < 2^-16, and then the neighbouring bf16 value."""
    a, b = got.double(), want.double()
    return (got.view(torch.int16) == want.view(torch.int16)) | (
        (a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16)
