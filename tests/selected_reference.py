"""Plain 64-bit definitions of the rotary and selected-block attention operators (torch)."""
import math

import torch

INF = math.inf


def rotary(x, positions, freqs, sections, rot, first, half, factor, inverse):
    axis = torch.tensor([a for a, p in enumerate(sections) for _ in range(p)], device=x.device)
    t = positions.double()[..., axis] * freqs
    c, s = factor * torch.cos(t)[:, None], factor * torch.sin(t)[:, None] * (-1 if inverse else 1)
    y = x.double().clone()
    part = y[..., first:first + rot]
    a, b = (part[..., :rot // 2], part[..., rot // 2:]) if half else (part[..., 0::2], part[..., 1::2])
    u, w = a * c - b * s, b * c + a * s
    y[..., first:first + rot] = torch.cat([u, w], -1) if half else torch.stack([u, w], -1).flatten(-2)
    return y


def means(k, block, lens):
    bt, h, n, d = k.shape
    out = torch.zeros(bt, h, -(-n // block), d, dtype=torch.float64, device=k.device)
    for i in range(bt):
        for g in range(out.shape[2]):
            m = min(int(lens[i]), (g + 1) * block) - g * block
            if m > 0:
                out[i, :, g] = k[i, :, g * block:g * block + m].double().sum(1) / m
    return out.float()


def visible(n, keys, lens, starts, causal, device):
    """[batch, n, keys]: keys that each query may see."""
    j = torch.arange(keys, device=device)
    ok = (j[None] < lens[:, None])[:, None, :].expand(-1, n, -1)
    if causal:
        pos = starts[:, None] + torch.arange(n, device=device)[None]
        ok = ok & (j[None, None] <= pos[..., None])
    return ok


def select(q, mean, keys, block, top, lens, starts, causal, n_first, n_local):
    bt, hq, n, d = q.shape
    hk, nb = mean.shape[1:3]
    sc = torch.einsum("bhnd,bhgd->bhng", q.double().unflatten(1, (hk, hq // hk)).sum(2), mean.double())
    sel = torch.full((bt, hk, n, top), -1, dtype=torch.int32)
    sc = sc.cpu()
    for b in range(bt):
        for i in range(n):
            pos = int(starts[b]) + i
            last = int(lens[b]) - 1
            if causal:
                last = min(last, pos)
            cand = 0 if last < 0 else last // block + 1
            forced = [g for g in range(cand) if g < n_first or (causal and pos // block - n_local < g <= pos // block)]
            for h in range(hk):
                row = sc[b, h, i].tolist()
                rest = sorted((g for g in range(cand) if g not in forced), key=lambda g: (-row[g], g))
                got = sorted((forced + rest)[:top])
                sel[b, h, i, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return sel.to(q.device)


def mask(sel, n, keys, block, lens, starts, causal):
    """[batch, key heads, n, keys] keys that each query attends to."""
    bt, hk = sel.shape[:2]
    nb = -(-keys // block)
    m = torch.zeros(bt, hk, n, nb + 1, dtype=torch.bool, device=sel.device)
    m.scatter_(3, torch.where(sel >= 0, sel, nb).long(), True)
    m = m[..., :nb].repeat_interleave(block, 3)[..., :keys]
    return m & visible(n, keys, lens, starts, causal, sel.device)[:, None]


def attention(q, k, v, ok, scale):
    """(out, lse, probabilities) in 64 bits; ok [batch, key heads, n, keys]."""
    grp = q.shape[1] // k.shape[1]
    live = ok.repeat_interleave(grp, 1)
    some = ok.any(2)[..., None]  # rows that no query attends to may hold anything
    kd = torch.where(some, k.double(), 0.0).repeat_interleave(grp, 1)
    vd = torch.where(some, v.double(), 0.0).repeat_interleave(grp, 1)
    x = torch.where(live, q.double() @ kd.transpose(2, 3) * scale, -INF)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m == -INF, 0.0, m))
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l > 0, l, 1.0)
    return p @ vd, (m + torch.log(l))[..., 0], p


def backward(dout, q, k, v, ok, scale, out=None):
    """(dq, dk, dv) and what bounds their errors; `out`: the rows that delta is formed from."""
    grp = q.shape[1] // k.shape[1]
    o, _, p = attention(q, k, v, ok, scale)
    some = ok.any(2)[..., None]
    kd = torch.where(some, k.double(), 0.0).repeat_interleave(grp, 1)
    vd = torch.where(some, v.double(), 0.0).repeat_interleave(grp, 1)
    g, qd = dout.double(), q.double()
    delta = (g * (o if out is None else out.double())).sum(-1, keepdim=True)
    ds = p * (g @ vd.transpose(2, 3) - delta) * scale
    wide = p * (g.abs() @ vd.abs().transpose(2, 3) + (g * o).abs().sum(-1, keepdim=True)) * scale

    def per_key(x):
        return x.unflatten(1, (k.shape[1], grp)).sum(2)

    grads = ds @ kd, per_key(ds.transpose(2, 3) @ qd), per_key(p.transpose(2, 3) @ g)
    sizes = ds.abs() @ kd.abs(), per_key(ds.abs().transpose(2, 3) @ qd.abs()), per_key(p.transpose(2, 3) @ g.abs())
    noise = wide @ kd.abs(), per_key(wide.transpose(2, 3) @ qd.abs()), sizes[2]
    return grads, sizes, noise
