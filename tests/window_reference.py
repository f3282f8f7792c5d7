"""Plain attention in 64 bits for rows that see any set of keys, with a bound on what the kernels' roundings
can do to each output.

`weight_unit` is half a step of the type in which the weights meet V (bf16: 2^-8, fp16: 2^-11).  As in
attn_reference.py, with W = sum_t w_t |v_t|: weights 2 u W / (1 - u), the output itself 2^-8 |out|, scores
4 ds W, sums 2 n 2^-24 W.  A cache in 8 bits adds, with s_t the scale of a token's values and T = 127 or 448:
  * INT8 codes enter the products as 1024 + 128 + q, whose 1152 is taken off again: what accumulates in fp32
    is then of the size of `k_size` = 1152 s (scores) and `v_size` = 1152 s (values) instead of |k| and |v|,
    one addition for each 16 keys on the way and 136 roundings around it;
  * a weight below the normal fp16 numbers is off by up to 2^-25 of the largest w_t s_t, times T.
"""
import torch

U = 2.0 ** -8


def attend(q, k, v, seen, weight_unit=U, k_size=None, v_size=None, v_scale=None, top=0.0):
    """q [n, 128], k, v [m, 128] float64; seen [n, m].  k_size [m] (or None: |k| itself), v_size [m],
    v_scale [m].  Returns (out, bound)."""
    n, m = q.shape[0], k.shape[0]
    if m == 0 or n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    root = 128.0 ** 0.5
    s = torch.where(seen, q @ k.T / root, -torch.inf)
    peak = s.max(dim=1, keepdim=True).values
    peak = torch.where(torch.isinf(peak), 0.0, peak)
    w = torch.exp(s - peak)
    l = w.sum(dim=1, keepdim=True)
    w = torch.where(l > 0, w / l, 0.0)
    out = w @ v
    weight = w @ v.abs()
    size = q.abs() @ k.abs().T
    if k_size is not None:
        size = size + q.abs().sum(dim=1, keepdim=True) * k_size[None, :]
    # (a query below the normal fp16 numbers is off by 2^-25)
    size = torch.where(seen, size + 2.0 ** -1 * k.abs().sum(dim=1)[None, :] * (weight_unit < U), 0.0) / root
    ds = 136 * 2.0 ** -24 * size.max(dim=1, keepdim=True).values + 2.0 ** -22
    rest = (2 * weight_unit / (1 - weight_unit) + 4 * ds + 2 * m * 2.0 ** -24) * weight
    if v_size is not None:
        rest = rest + (m / 16 + 136) * 2.0 ** -23 * (w @ v_size)[:, None]
    if v_scale is not None:
        rest = rest + m * 2.0 ** -25 * top * (w * v_scale[None, :]).max(dim=1, keepdim=True).values
    return out, rest + U * (out.abs() + rest)


def visible(positions, m, window, sinks):
    """[n, m]: whether the row at positions[i] sees key t (window 0: all up to its own)."""
    p, t = positions[:, None], torch.arange(m)[None, :]
    causal = t <= p
    return causal if window == 0 else causal & ((t > p - window) | (t < sinks))
