"""Attention of packed rows over a paged cache in float64, a request's rows of
one cache head at a time (the oracle takes a row and a head at a time, too
slow for thousands of tokens and rows), with the terms of an error bound."""
import numpy as np
import torch


def attend64(q, kc, vc, table, length, K, offs, *, causal=True, scale, k_scale=None, v_scale=None):
    """(out, lse, mean, ds): the exact rows and log-sum-exps, the weighted
    means of |v|, and what bounds the error of any score of a row formed as a
    float32 sum of D exact products: (D + 4) 2^-24 scale max |k_scale k| . |q|."""
    n_rows, Hq, D = q.shape
    page, H = kc.shape[1:3]
    group = Hq // H
    f64 = lambda x: x.detach().to("cpu").to(torch.float32).to(torch.float64)
    q, kc, vc = f64(q), kc.detach().cpu(), vc.detach().cpu()
    one = torch.ones(H, dtype=torch.float64)
    ks, vs = one if k_scale is None else f64(k_scale), one if v_scale is None else f64(v_scale)
    out, mean = [torch.full((n_rows, Hq, D), float("nan"), dtype=torch.float64) for _ in range(2)]
    lse, ds = [torch.full((n_rows, Hq), float("nan"), dtype=torch.float64) for _ in range(2)]
    for b in range(len(K)):
        n_b, L = int(K[b]) + 1, int(length[b] + K[b]) + 1
        if n_b < 1:
            continue
        t = np.arange(L)
        ids = torch.from_numpy(np.asarray(table[b])[t // page].astype(np.int64))
        at = torch.from_numpy(t % page)
        rows = slice(int(offs[b]), int(offs[b]) + n_b)
        sees = torch.from_numpy(length[b] + np.arange(n_b) if causal else np.full(n_b, L - 1))
        hidden = (torch.arange(L)[None, :] > sees[:, None]).repeat_interleave(group, 0)
        for h in range(H):
            k, v = f64(kc[ids, at, h]) * ks[h], f64(vc[ids, at, h]) * vs[h]
            x = q[rows, h * group:(h + 1) * group].reshape(n_b * group, D)
            s = (scale * (x @ k.T)).masked_fill(hidden, -float("inf"))
            top = s.max(1, keepdim=True).values
            e = torch.exp(s - top)
            sums = e.sum(1, keepdim=True)
            put = lambda y: y.reshape(n_b, group, -1)
            to = slice(h * group, (h + 1) * group)
            out[rows, to], mean[rows, to] = put(e @ v / sums), put(e @ v.abs() / sums)
            lse[rows, to] = put(top + sums.log())[..., 0]
            ds[rows, to] = put((D + 4) * 2.0 ** -24 * scale * (x.abs() @ k.abs().max(0).values)[:, None])[..., 0]
    return out.numpy(), lse.numpy(), mean.numpy(), ds.numpy()


def worst_error(s, out, lse, causal, weight, floor=0.0):
    """The largest error over its bound.  A result o = sum p v / sum p with A =
    sum p |v| / sum p is rounded to bf16 (2^-8 |o|); a weight is rounded by
    ``weight`` of it and ``floor`` of the largest; weights are off by 2 ds + n
    2^-24 + 2^-20 besides (scores, float32 sums of n terms, a few units of the
    hardware exponential)."""
    want, wl, mean, ds = attend64(s["q"], s["kc"], s["vc"], s["table"], s["length"], s["K"], s["offs"], causal=causal,
                                  scale=s["scale"], k_scale=s["ks"], v_scale=s["vs"])
    n = int((s["length"] + s["K"]).max()) + 1
    vmax = s["vc"].float().abs().max().item() * (1.0 if s["vs"] is None else s["vs"].max().item())
    tol = 2.0 ** -8 * np.abs(want) + (weight + 2 * ds[..., None] + n * 2.0 ** -24 + 2.0 ** -20) * mean + n * floor * vmax
    there = ~np.isnan(want[:, 0, 0])
    err = np.abs(out.float().cpu().double().numpy() - want)[there]
    assert np.isfinite(err).all()
    el = np.abs(lse.cpu().double().numpy() - wl)[there] / (ds + n * 2.0 ** -24 + 2.0 ** -20 * (1 + np.abs(wl)))[there]
    return max((err / tol[there]).max(), el.max())
