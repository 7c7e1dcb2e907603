"""64-bit definitions of the rotary, shared-prefix, entry-weight and eviction
operators, with error bounds of the kernels' arithmetic (shared by the tests)."""
import math

import torch

EPS32 = 2.0 ** -24                       # half a step of fp32


def half_step(dt) -> float:
    return torch.finfo(dt).eps / 2


# ------------------------------------------------------------------ rotary
def rope(x, pos, freqs, off, interleaved, scale, transpose):
    """(result, bound) in float64; x [B, n, H, D], pos [B, n] (negative: unrotated)."""
    v = x.double()
    rot = 2 * freqs.numel()
    ang = pos.double()[:, :, None, None] * freqs.to(x.device)
    if transpose:
        ang = -ang
    r = v[..., off:off + rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :rot // 2], r[..., rot // 2:])
    u, w = scale * (a * ang.cos() - b * ang.sin()), scale * (b * ang.cos() + a * ang.sin())
    mag = scale * (a.abs() + b.abs())
    join = (lambda p, q: torch.stack([p, q], -1).flatten(-2)) if interleaved else \
        (lambda p, q: torch.cat([p, q], -1))
    res, bound = v.clone(), torch.zeros_like(v)
    res[..., off:off + rot] = join(u, w)
    # cos and sin: the angle within pi 2^-25 (its fp32 form, in units of pi) + 2 pi 2^-32 (64-bit
    # phase cut to 32) and sincospi within 2 ulp (2^-23), times scale (2^-24): 2.8e-7; the two
    # products and the sum: 3 roundings of 2^-24 (1.8e-7)
    bound[..., off:off + rot] = join(mag, mag) * 4.6e-7
    bound += half_step(x.dtype) * res.abs()
    void = (pos < 0)[:, :, None, None].expand_as(v)
    res = torch.where(void, v, res)
    bound = torch.where(void, torch.zeros_like(v), bound)
    bound[..., :off] = 0
    bound[..., off + rot:] = 0
    return res, bound


# ------------------------------------------------------------------ attention
def attention_row(q, keys, scale, dt, p_bits_dt=None):
    """One query row q [H, D] over keys [n, D] (float64): (out, lse, out bound, lse bound).
    ``p_bits_dt``: the type the kernel rounds its softmax weights to (None: fp32)."""
    H, D = q.shape
    if keys.shape[0] == 0:
        z = torch.zeros(H, D, dtype=torch.float64, device=q.device)
        return z, torch.full((H,), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0]
    s = scale * (q @ keys.t())
    mag = scale * (q.abs() @ keys.abs().t())
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out = p @ keys
    # a score: D products and sums in fp32, the scale and log2(e) factors, the subtraction of the
    # running maximum, 2^x within 2^-22
    dz = (D + 4) * EPS32 * mag + 4 * EPS32 * (s.abs() + lse.abs()[:, None]) + 2.0 ** -22
    n = keys.shape[0]
    dp = dz + (half_step(p_bits_dt) if p_bits_dt else 0.0)
    # the weights enter numerator and denominator: each relative change moves the result by at
    # most p |v| + p |out|; the sums of n terms add n roundings at most
    spread = (p * dp) @ keys.abs() + (p * dp).sum(-1, keepdim=True) * out.abs()
    bound = spread * 1.01 + 2 * (n + 8) * EPS32 * (p @ keys.abs()) + half_step(dt) * out.abs() * 1.01
    dl = (p * dz).sum(-1) + (n + 8) * EPS32 + 4 * EPS32 * lse.abs()
    return out, lse, bound, dl


def prefix_attention(a, dt, p_bits_dt=None):
    """``a``: dict(q, kv_p, kv_c, m, kv_raw, window, n_entries, raw_pos0, raw_len, q_pos), the
    optional arrays None; returns (out, lse, out bound, lse bound) over [B, n_q, H(, D)]."""
    q = a["q"]
    B, nq, H, D = q.shape
    Np, cap, L = a["kv_p"].shape[0], a["kv_c"].shape[1], a["kv_raw"].shape[1]
    scale = a.get("scale") or D ** -0.5
    res = [torch.empty(B, nq, H, D, dtype=torch.float64, device=q.device) for _ in range(2)]
    ls = [torch.empty(B, nq, H, dtype=torch.float64, device=q.device) for _ in range(2)]
    get = lambda k, b, d: d if a.get(k) is None else int(a[k][b])  # noqa: E731
    for b in range(B):
        ne = min(max(get("n_entries", b, Np + cap), 0), Np + cap)
        p0, ln = get("raw_pos0", b, 0), min(max(get("raw_len", b, L), 0), L)
        for j in range(nq):
            t = j if a.get("q_pos") is None else int(a["q_pos"][b, j])
            vis = min((t + 1) // a["m"], ne) if t >= 0 else 0
            rows = [i for i in range(ln) if p0 + i >= 0 and t - a["window"] < p0 + i <= t]
            keys = torch.cat([a["kv_p"][:min(vis, Np)], a["kv_c"][b, :max(vis - Np, 0)],
                              a["kv_raw"][b, rows]]).double()
            o, l, bo, bl = attention_row(q[b, j].double(), keys, scale, dt, p_bits_dt)
            res[0][b, j], res[1][b, j], ls[0][b, j], ls[1][b, j] = o, bo, l, bl
    return res[0], ls[0], res[1], ls[1]


# ------------------------------------------------------------------ entry weights
def entry_weights(q, kv, m, lse, weight_in, idx, n_entries, q_pos, scale=None):
    """(weights, bound) in float64."""
    B, nq, H, D = q.shape
    N = kv.shape[1]
    scale = scale or D ** -0.5
    w = torch.zeros(B, N, dtype=torch.float64, device=q.device) if weight_in is None else weight_in.double()
    bound = EPS32 * w.abs()
    for b in range(B):
        ne = N if n_entries is None else min(max(int(n_entries[b]), 0), N)
        listed = list(range(N)) if idx is None else [int(s) for s in idx[b] if 0 <= int(s) < N]
        for j in range(nq):
            t = j if q_pos is None else int(q_pos[b, j])
            vis = min((t + 1) // m, ne) if t >= 0 else 0
            s = torch.tensor([i for i in listed if i < vis], dtype=torch.long, device=q.device)
            live = lse[b, j] > -math.inf
            if not len(s) or not bool(live.any()):
                continue
            k, qq, ll = kv[b, s].double(), q[b, j][live].double(), lse[b, j][live].double()
            z = scale * (k @ qq.t())
            p = torch.exp(z - ll)
            mag = scale * (k.abs() @ qq.abs().t())
            dz = (D + 4) * EPS32 * mag + 4 * EPS32 * (z.abs() + ll.abs()) + 2.0 ** -22
            w[b].index_add_(0, s, p.sum(1))
            bound[b].index_add_(0, s, (p * (dz + (nq * H + 8) * EPS32)).sum(1))
    return w, bound * 1.01 + 2 * EPS32 * w.abs() + 1e-37


# ------------------------------------------------------------------ eviction
def evict(weight, n_entries, budget, recent):
    """(idx, n_kept, weight) as lists / a tensor on the CPU."""
    w = weight.cpu().clone()
    B, N = w.shape
    idx = torch.full((B, budget), -1, dtype=torch.int32)
    kept = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        V = N if n_entries is None else min(max(int(n_entries[b]), 0), N)
        row = w[b].tolist()
        fit = [s for s in range(V) if row[s] >= 0]
        new = sorted((s for s in fit if s >= V - recent), reverse=True)
        old = sorted((s for s in fit if s < V - recent), key=lambda s: (-row[s], s))
        keep = sorted((new + old)[:budget])
        idx[b, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
        kept[b] = len(keep)
        gone = torch.ones(V, dtype=torch.bool)
        gone[keep] = False
        w[b, :V][gone] = -1.0
    return idx, kept, w
