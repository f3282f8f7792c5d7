"""Plain attention in 64 bits for the tests of the bf16 operators, with a bound on what their roundings
can do to each output.

The bound, per output element (u = 2^-8, half a step of bf16 relative to the value; W = sum_t w_t |v_t|
over the softmax weights w):
  * weights rounded to bf16 before they meet V: each w_t is off by a factor 1 + e, |e| <= u, so the sum
    is off by at most u W; where the normalising sum is of the rounded weights too, it is off by at most
    a factor 1 + u itself: 2 u W / (1 - u) covers both ways of summing;
  * the output rounded to bf16: u |out| (of the computed value, hence of |out| plus the rest);
  * scores accumulated in fp32 over 128 products, scaled, offset by the maximum and raised to a power:
    |ds| <= (128 + 8) 2^-24 A with A = sum_d |q_d k_d| / sqrt(128) for the accumulation and the
    roundings around it, plus 2^-22 for the exponential itself: each weight and the sum move by at most
    e^ds - 1 <= 2 ds (ds < 1), hence 4 ds W;
  * sums of weights and of weighted values in fp32 over n keys: 2 n 2^-24 W.
"""
import torch

U = 2.0 ** -8


def attend(q, k, v, lim):
    """q [n, 128], k, v [m, 128] float64; lim [n]: row i sees keys t < lim[i].  Returns (out, bound)."""
    n, m = q.shape[0], k.shape[0]
    if m == 0 or n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    seen = torch.arange(m)[None, :] < lim[:, None]
    s = q @ k.T / 128.0 ** 0.5
    s = torch.where(seen, s, torch.full_like(s, -torch.inf))
    top = s.max(dim=1, keepdim=True).values
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(s - top)
    l = w.sum(dim=1, keepdim=True)
    w = torch.where(l > 0, w / l, torch.zeros_like(w))
    out = w @ v
    weight = w @ v.abs()
    a = torch.where(seen, q.abs() @ k.abs().T / 128.0 ** 0.5, torch.zeros_like(s)).max(dim=1, keepdim=True).values
    ds = 136 * 2.0 ** -24 * a + 2.0 ** -22
    rest = (2 * U / (1 - U) + 4 * ds + 2 * m * 2.0 ** -24) * weight
    return out, rest + U * (out.abs() + rest)


def prompt(q, ks, vs, q_lens, hq, hkv):
    """q [Tq, hq, 128]; ks, vs per request [m, hkv, 128] (CPU tensors).  Returns (out, bound)."""
    g = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros(q.shape, dtype=torch.float64)
    at = 0
    for n, k, v in zip(q_lens, ks, vs):
        m = k.shape[0]
        lim = (m - n + torch.arange(n) + 1).clamp(min=0)
        for h in range(hq):
            o, e = attend(q[at:at + n, h].double(), k[:, h // g].double(), v[:, h // g].double(), lim)
            out[at:at + n, h], bound[at:at + n, h] = o, e
        at += n
    return out, bound


def check(got, ref, bound):
    got = got.cpu().double()
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() > bound
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} outside the bound, first at {i}: got {got[i]:.6g} "
                             f"ref {ref[i]:.6g} bound {bound[i]:.3g}; max |diff| {(got - ref).abs().max():.3g}")


class Pages:
    """ks, vs (per request [m, hkv, 128] bf16 on the CPU) laid out in shuffled bf16 pages; every slot
    that no token owns, spare pages and unused table entries among them, holds `fill`."""

    def __init__(self, ks, vs, hkv, block, seed=0, extra=3, spare_columns=1, fill=float("nan")):
        g = torch.Generator().manual_seed(seed)
        need = [(k.shape[0] + block - 1) // block for k in ks]
        total = sum(need) + extra
        order = torch.randperm(total, generator=g).to(torch.int32)
        self.table = torch.full((len(ks), max(need) + spare_columns), int(order[-1]), dtype=torch.int32)
        self.k = torch.full((total, hkv, block, 128), fill, dtype=torch.bfloat16)
        self.v = self.k.clone()
        at = 0
        for b, (k, v) in enumerate(zip(ks, vs)):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            t = torch.arange(k.shape[0])
            page = self.table[b].long()[t // block]
            self.k[page, :, t % block] = k
            self.v[page, :, t % block] = v
        self.lens = torch.tensor([k.shape[0] for k in ks], dtype=torch.int32)
        self.need = need

    def cuda(self):
        for n in ("k", "v", "table", "lens"):
            setattr(self, n, getattr(self, n).cuda())
        return self


def rows(n, heads, seed, sigma=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, 128, generator=g) * sigma).to(torch.bfloat16)
