"""Cases and plain forms of the long-context serving operators around HCA decode.

Four operators that a serving loop runs next to the compressed attention:

``rope``     rotary positions of the query heads and the shared-KV row (part of
             the head rotated, interleaved or half layout, YaRN-scaled
             frequencies), forward and transposed (gradient, or taking the
             position out of an attention output);
``prefix``   HCA attention for a batch whose elements share their first N_p
             compressed entries: those are stored once, each element adds its
             own entries and its sliding window, under one softmax;
``weights``  the attention weight that each compressed entry received, summed
             over heads and query rows and added to what it had before;
``evict``    the entries that a cache of a given budget keeps: the most recent
             ones and, of the rest, those of largest accumulated weight.

``run`` computes them in plain torch operations, or, where ``own`` is set,
through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of 64 sequences at contexts up to 128K: latency only
        dict(name="rope decode b64", op="rope", dt="bf16", B=64, n=1, H=64, Hy=1, D=128, rot=64, off=64,
             layout="interleaved", far=131072, factor=16.0, transpose=False, fused=False),
        # the prompt of two sequences of 8192 tokens
        dict(name="rope prefill 2x8192", op="rope", dt="bf16", B=2, n=8192, H=64, Hy=1, D=128, rot=64, off=64,
             layout="half", far=8192, factor=1.0, transpose=False, fused=False),
        # gradient of the rotation, fp32, a ragged length, heads cut out of a fused projection
        dict(name="rope gradient f32 3x509", op="rope", dt="f32", B=3, n=509, H=8, Hy=2, D=64, rot=64, off=0,
             layout="half", far=1048576, factor=4.0, transpose=True, fused=True),
        # two users of one 128K system prompt: the smallest decode call
        dict(name="prefix decode b2 128K", op="prefix", dt="bf16", B=2, nq=1, H=64, D=128, m=128, Np=1024, own=16,
             window=512, pad=False),
        # 64 users of one 1M-token document
        dict(name="prefix decode b64 1M", op="prefix", dt="bf16", B=64, nq=1, H=64, D=128, m=128, Np=8192, own=64,
             window=512, pad=False),
        # a ragged batch of 3-token drafts over a prefix that ends inside a tile, one slot of the batch empty
        dict(name="prefix draft b67x3 ragged", op="prefix", dt="bf16", B=67, nq=3, H=64, D=128, m=128, Np=4099, own=77,
             window=509, pad=True),
        # fp32 with the small head layout
        dict(name="prefix decode f32 b5", op="prefix", dt="f32", B=5, nq=2, H=8, D=64, m=4, Np=509, own=33, window=32,
             pad=False),
        # one decode step of 16 sequences at 1M tokens
        dict(name="weights decode b16 1M", op="weights", dt="bf16", B=16, nq=1, H=64, D=128, m=128, N=8192, keep=0),
        # the last 64 queries of a 64K prompt look over all its entries
        dict(name="weights prompt tail 64K", op="weights", dt="bf16", B=1, nq=64, H=64, D=128, m=4, N=16384, keep=0),
        # decode over the lists of kept entries, after an eviction
        dict(name="weights kept b64x1999", op="weights", dt="bf16", B=64, nq=1, H=64, D=128, m=128, N=8192, keep=1999),
        # the caches of 64 sequences cut to 2048 entries each
        dict(name="evict b64 32K to 2K", op="evict", B=64, N=32768, budget=2048, recent=128, again=False),
        # a small ragged cache that was cut before
        dict(name="evict b3 777 to 100", op="evict", B=3, N=777, budget=100, recent=7, again=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prefix", "weights", "evict"])
    if op == "rope":
        dt, D = rng.choice(["bf16", "bf16", "f32"]), rng.choice([32, 64, 80, 128, 192, 256])
        H, B = rng.choice([1, 4, 8, 16, 64]), rng.randint(1, 64)
        rot = min(D, rng.choice([16, 32, 50, 64, 128]))
        most = 2 * 8192 * 64 * 128 * 2 // (H * D * (2 if dt == "bf16" else 4))
        return dict(op=op, dt=dt, B=B, n=_log(rng, 1, max(1, min(most // B // 4, 8192))), H=H, Hy=rng.choice([0, 1, 2]),
                    D=D, rot=rot, off=rng.choice([0, D - rot]), layout=rng.choice(["half", "interleaved"]),
                    far=_log(rng, 1000, 1048576), factor=rng.choice([1.0, 4.0, 16.0, 40.0]),
                    transpose=rng.random() < 0.4, fused=rng.random() < 0.3)
    if op == "prefix":
        if rng.random() < 0.2:
            return dict(op=op, dt="f32", B=rng.randint(1, 9), nq=rng.randint(1, 3), H=rng.choice([8, 16]), D=64,
                        m=rng.choice([4, 128]), Np=_log(rng, 1, 1000), own=rng.randint(0, 100),
                        window=_log(rng, 1, 128), pad=rng.random() < 0.3)
        nq, H = rng.choice([1, 1, 1, 2, 3, 4]), rng.choice([64, 64, 64, 128])
        return dict(op=op, dt="bf16", B=_log(rng, 1, 80 * 64 // H // nq), nq=nq, H=H, D=128, m=rng.choice([4, 128]),
                    Np=_log(rng, 64, 5000), own=rng.choice([0, rng.randint(1, 150)]), window=_log(rng, 16, 512),
                    pad=rng.random() < 0.3)
    if op == "weights":
        dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
        nq = rng.choice([1, 1, 2, rng.randint(3, 64)])
        N = _log(rng, 32, 8192 if dt == "bf16" else 1024)
        B = rng.randint(1, max(1, min(32, 64 * 16384 // (nq * N))) if dt == "bf16" else 4)
        keep = rng.choice([0, 0, rng.randint(1, min(N, 2048))])
        return dict(op=op, dt=dt, B=B, nq=nq, H=rng.choice([64, 128, 16]) if dt == "bf16" else 8,
                    D=128 if dt == "bf16" else 64, m=rng.choice([4, 128]), N=N, keep=keep)
    N = _log(rng, 1, 32768)
    return dict(op=op, B=rng.randint(1, 64), N=N, budget=_log(rng, 1, max(1, min(N, 4096))), recent=rng.choice([0, 1, rng.randint(2, 300)]),
                again=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, dt, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(dt)


def _ints(g, lo, hi, *shape):
    """Whole numbers in [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int32)


def _yarn(rot, factor, base=10000.0, original=65536, fast=32.0, slow=1.0):
    """Frequencies (radians a position) of the rotated pairs and the factor on cos and sin: pairs that turn more than `fast`
    times within `original` positions keep their frequency, those below `slow` turns are slowed down by `factor`, and a
    linear ramp over the pairs joins the two."""
    f = [base ** (-2.0 * j / rot) for j in range(rot // 2)]
    if factor <= 1.0:
        return f, 1.0
    pair_of = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), rot - 1)
    hi = hi if hi > lo else lo + 0.001
    keep = [1.0 - min(max((j - lo) / (hi - lo), 0.0), 1.0) for j in range(rot // 2)]
    return [v / factor * (1 - k) + v * k for v, k in zip(f, keep)], 0.1 * math.log(factor) + 1.0


def _prepare_rope(c, g):
    dt, B, n, D = TYPES[c["dt"]], c["B"], c["n"], c["D"]
    if c["fused"]:   # heads as they leave a fused projection: a slice of [B, n, (H + Hy + 1) * D]
        all_ = _normal(g, dt, B, n, c["H"] + c["Hy"] + 1, D)
        x, y = all_[:, :, :c["H"]], all_[:, :, c["H"]:c["H"] + c["Hy"]]
    else:
        x, y = _normal(g, dt, B, n, c["H"], D), _normal(g, dt, B, n, c["Hy"], D)
    start = _ints(g, 0, max(0, c["far"] - n), B, 1)
    pos = (start + torch.arange(n, device=DEV, dtype=torch.int32)).contiguous()
    if n > 4 and B > 1:   # the last element's prompt is shorter than the batch's
        pos[-1, n - n // 4:] = -1
    freqs, scale = _yarn(c["rot"], c["factor"])
    return dict(x=x, y=y if c["Hy"] else None, pos=pos, freqs=torch.tensor(freqs, dtype=torch.float64), scale=scale)


def _prepare_prefix(c, g):
    dt, B, nq, H, D, m = TYPES[c["dt"]], c["B"], c["nq"], c["H"], c["D"], c["m"]
    L = c["window"] + nq - 1
    own_n = _ints(g, 0, c["own"], B)
    last = (c["Np"] + own_n) * m + _ints(g, 0, m - 1, B) - 1 + nq * m   # every query sees the whole prefix
    q_pos = last[:, None] - (nq - 1) + torch.arange(nq, device=DEV, dtype=torch.int32)
    if c["pad"] and B > 1:
        q_pos[-1] = -1
    return dict(q=_normal(g, dt, B, nq, H, D), kv_p=_normal(g, dt, c["Np"], D), kv_c=_normal(g, dt, B, c["own"], D),
                kv_raw=_normal(g, dt, B, L, D), n_entries=(c["Np"] + own_n).contiguous(), q_pos=q_pos.contiguous(),
                raw_pos0=(last - (L - 1)).contiguous(), raw_len=torch.full((B,), L, device=DEV, dtype=torch.int32))


def _prepare_weights(c, g):
    dt, B, nq, H, D, m, N = TYPES[c["dt"]], c["B"], c["nq"], c["H"], c["D"], c["m"], c["N"]
    q, kv = _normal(g, dt, B, nq, H, D), _normal(g, dt, B, N, D)
    n_entries = _ints(g, (N + 1) // 2, N, B)
    q_pos = ((n_entries * m + m - 2)[:, None] - (nq - 1) + torch.arange(nq, device=DEV, dtype=torch.int32)).contiguous()
    idx = None
    seen = torch.arange(N, device=DEV) < torch.minimum((q_pos + 1) // m, n_entries[:, None])[..., None]   # [B, nq, N]
    if c["keep"]:
        order = torch.rand(B, N, generator=g, device=DEV).argsort(1)[:, :c["keep"]].sort(1)[0].to(torch.int32)
        short = torch.arange(c["keep"], device=DEV) >= c["keep"] - (torch.arange(B, device=DEV) % 3)[:, None]
        idx = torch.where(short, -1, order).contiguous()   # two lists of three end in padding
        listed_ = torch.zeros(B, N + 1, dtype=torch.bool, device=DEV)
        listed_.scatter_(1, torch.where(idx < 0, N, idx).long(), True)
        seen = seen & listed_[:, None, :N]
    lse = torch.empty(B, nq, H, device=DEV)
    for b in range(B):   # the attention's own lse: these entries and a window of half their mass
        z = q[b].float().reshape(nq * H, D) @ kv[b].float().t() / math.sqrt(D)
        z = z.reshape(nq, H, N).masked_fill(~seen[b][:, None], -math.inf)
        lse[b] = torch.logaddexp(torch.logsumexp(z, -1), torch.tensor(math.log(1 + N / 2), device=DEV))
    return dict(q=q, kv=kv, lse=lse, weight=torch.rand(B, N, generator=g, device=DEV) * (nq * H / N), n_entries=n_entries, q_pos=q_pos, idx=idx)


def _prepare_evict(c, g):
    B, N = c["B"], c["N"]
    w = torch.rand(B, N, generator=g, device=DEV).log().neg()   # a few heavy entries, many light ones
    w = torch.where(torch.rand(B, N, generator=g, device=DEV) < 0.05, torch.zeros_like(w), w)   # some never looked at
    w = torch.where(torch.rand(B, N, generator=g, device=DEV) < 0.3, (w * 16).round() / 16, w)   # and equal ones
    if c["again"]:
        w = torch.where(torch.rand(B, N, generator=g, device=DEV) < 0.4, torch.full_like(w, -1), w)
    return dict(weight=w.contiguous(), n_entries=_ints(g, N // 2, N, B))


def prepare(case, seed):
    state = globals()["_prepare_" + case["op"]](case, _gen(seed))
    state["case"] = dict(case)
    return state


# ------------------------------------------------------------------ the operators, plain
def _rope_plain(s):
    c = s["case"]
    half, off = c["rot"] // 2, c["off"]
    angle = s["pos"].double()[..., None] * s["freqs"].to(DEV)
    cos, sin = (angle.cos() * s["scale"]).float()[:, :, None], (angle.sin() * s["scale"]).float()[:, :, None]
    if c["transpose"]:
        sin = -sin
    void = (s["pos"] < 0)[:, :, None, None]

    def turn(x):
        if x is None:
            return None
        v = x.float()
        r = v[..., off:off + c["rot"]]
        a, b = (r[..., :half], r[..., half:]) if c["layout"] == "half" else (r[..., 0::2], r[..., 1::2])
        u, w = a * cos - b * sin, b * cos + a * sin
        r = torch.cat([u, w], -1) if c["layout"] == "half" else torch.stack([u, w], -1).flatten(-2)
        return torch.where(void, v, torch.cat([v[..., :off], r, v[..., off + c["rot"]:]], -1)).to(x.dtype)

    return turn(s["x"]), turn(s["y"])


def _prefix_plain(s):
    c = s["case"]
    q, kp, kc, kr = (s[k].float() for k in ("q", "kv_p", "kv_c", "kv_raw"))
    B, nq, H, D = q.shape
    t = s["q_pos"][..., None]
    vis = torch.minimum((t + 1) // c["m"], s["n_entries"][:, None, None])
    place = s["raw_pos0"][:, None, None] + torch.arange(kr.shape[1], device=DEV)
    seen = torch.cat([torch.arange(c["Np"], device=DEV) < vis, c["Np"] + torch.arange(c["own"], device=DEV) < vis,
                      (place >= 0) & (place <= t) & (place > t - c["window"])], -1) & (t >= 0)
    rows = q.reshape(B, nq * H, D)
    z = torch.cat([rows.reshape(-1, D).matmul(kp.t()).reshape(B, nq * H, -1), rows.matmul(kc.mT), rows.matmul(kr.mT)], -1)
    z = (z / math.sqrt(D)).reshape(B, nq, H, -1).masked_fill(~seen[:, :, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = (z - top.masked_fill(top == -math.inf, 0)).exp()
    total = p.sum(-1, keepdim=True)
    p = p.reshape(B, nq * H, -1)
    o = p[..., :c["Np"]].reshape(B * nq * H, -1).matmul(kp).reshape(B, nq * H, D)
    o = o + p[..., c["Np"]:c["Np"] + c["own"]].matmul(kc) + p[..., c["Np"] + c["own"]:].matmul(kr)
    o = o.reshape(B, nq, H, D) / total.masked_fill(total == 0, 1)
    return o.to(s["q"].dtype), (top + total.log()).squeeze(-1)


def _weights_plain(s):
    c = s["case"]
    q, kv, (B, nq, H, D) = s["q"].float(), s["kv"].float(), s["q"].shape
    vis = torch.minimum((s["q_pos"] + 1) // c["m"], s["n_entries"][:, None])[..., None]
    if s["idx"] is None:
        z = q.reshape(B, nq * H, D).matmul(kv.mT) / math.sqrt(D)
        p = (z.reshape(B, nq, H, -1) - s["lse"][..., None]).exp()
        return s["weight"] + (p * (torch.arange(c["N"], device=DEV) < vis)[:, :, None]).sum((1, 2))
    at = s["idx"].clamp(min=0).long()
    rows = kv.gather(1, at[..., None].expand(-1, -1, D))
    z = q.reshape(B, nq * H, D).matmul(rows.mT) / math.sqrt(D)
    p = (z.reshape(B, nq, H, -1) - s["lse"][..., None]).exp()
    seen = (s["idx"][:, None] >= 0) & (s["idx"][:, None] < vis)
    return s["weight"].scatter_add(1, at, (p * seen[:, :, None]).sum((1, 2)))


def _evict_plain(s):
    c, w = s["case"], s["weight"]
    place = torch.arange(c["N"], device=DEV)
    inside = place < s["n_entries"][:, None]
    fit = inside & (w >= 0)
    fresh = fit & (place >= s["n_entries"][:, None] - c["recent"])
    rank = torch.where(fresh, -place, 1)   # newest first, before all others
    by_weight = torch.where(fit, w, -1.0).sort(dim=1, descending=True, stable=True)[1]
    order = by_weight.gather(1, rank.gather(1, by_weight).sort(dim=1, stable=True)[1])
    first = order[:, :c["budget"]]
    kept = torch.zeros_like(inside).scatter(1, first, fit.gather(1, first))
    idx = torch.where(kept, place, c["N"]).sort(1)[0][:, :c["budget"]]
    w.copy_(torch.where(inside & ~kept, -1.0, w))
    return torch.where(idx < c["N"], idx, -1).to(torch.int32), kept.sum(1).to(torch.int32), w


def _own(s):
    from long_context_compressed_03_b200 import api
    c = s["case"]
    if c["op"] == "rope":
        return api.rope(s["x"], s["freqs"], pos=s["pos"], y=s["y"], rot_offset=c["off"], interleaved=c["layout"] == "interleaved",
                        scale=s["scale"], transpose=c["transpose"])
    if c["op"] == "prefix":
        return api.hca_attn_prefix(s["q"], s["kv_p"], s["kv_c"], c["m"], s["kv_raw"], c["window"], with_lse=True,
                                   n_entries=s["n_entries"], raw_pos0=s["raw_pos0"], raw_len=s["raw_len"], q_pos=s["q_pos"])
    if c["op"] == "weights":
        return api.entry_weights(s["q"], s["kv"], c["m"], s["lse"], weight=s["weight"], idx=s["idx"], n_entries=s["n_entries"],
                                 q_pos=s["q_pos"])
    return *api.evict(s["weight"], c["budget"], recent=c["recent"], n_entries=s["n_entries"]), s["weight"]


def run(state):
    if own:
        return _own(state)
    return globals()["_" + state["case"]["op"] + "_plain"](state)


# ------------------------------------------------------------------ what they cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        rows = c["B"] * c["n"] * (c["H"] + c["Hy"])
        return dict(bytes=2 * rows * c["D"] * TYPES[c["dt"]].itemsize + 4 * c["B"] * c["n"], flops=3 * rows * c["rot"])
    if c["op"] == "prefix":
        size, rows = TYPES[c["dt"]].itemsize, c["B"] * c["nq"] * c["H"]
        keys = c["Np"] + c["own"] / 2 + c["window"]
        read = 2 * rows * c["D"] + c["Np"] * c["D"] + c["B"] * (c["own"] / 2 + c["window"] + c["nq"] - 1) * c["D"]
        return dict(bytes=size * read + 4 * rows, flops=4 * rows * c["D"] * keys)
    if c["op"] == "weights":
        size, rows = TYPES[c["dt"]].itemsize, c["nq"] * c["H"]
        keys = c["keep"] * 0.75 if c["keep"] else 0.75 * c["N"]
        return dict(bytes=c["B"] * (size * (rows + keys) * c["D"] + 4 * rows + 8 * c["N"] + 4 * c["keep"]),
                    flops=2 * c["B"] * rows * c["D"] * keys)
    return dict(bytes=c["B"] * (4 * 0.75 * c["N"] * 2 + 4 * c["budget"] + 8), flops=c["B"] * c["N"])


# ------------------------------------------------------------------ the definitions in 64 bits
def _rope_exact(s):
    c, out = s["case"], []
    turn = torch.polar(torch.full_like(s["pos"].double(), s["scale"])[..., None] + 0 * s["freqs"].to(DEV),
                       s["pos"].double()[..., None] * s["freqs"].to(DEV))
    turn = turn.conj() if c["transpose"] else turn
    for x in (s["x"], s["y"]):
        if x is None:
            out.append(None)
            continue
        v = x.double().contiguous()
        mid = v[..., c["off"]:c["off"] + c["rot"]]
        pairs = mid.unflatten(-1, (2, -1)).transpose(-1, -2) if c["layout"] == "half" else mid.unflatten(-1, (-1, 2))
        r = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, :, None])
        w = v.clone()
        w[..., c["off"]:c["off"] + c["rot"]] = (r.transpose(-1, -2) if c["layout"] == "half" else r).flatten(-2)
        w[s["pos"] < 0] = v[s["pos"] < 0]
        out.append(w)
    return tuple(out)


def _prefix_exact(s):
    c = s["case"]
    out, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.full(s["q"].shape[:3], -math.inf, dtype=torch.float64, device=DEV)
    pos, n, p0, ln = (s[k].tolist() for k in ("q_pos", "n_entries", "raw_pos0", "raw_len"))
    for b in range(c["B"]):
        cache = torch.cat([s["kv_p"], s["kv_c"][b]]).double()
        for j in range(c["nq"]):
            t = pos[b][j]
            if t < 0:
                continue
            lo, hi = max(0, t - c["window"] + 1) - p0[b], min(t - p0[b] + 1, ln[b])
            keys = torch.cat([cache[:min((t + 1) // c["m"], n[b])], s["kv_raw"][b, max(lo, 0):max(hi, 0)].double()])
            z = s["q"][b, j].double() @ keys.t() * c["D"] ** -0.5
            if keys.shape[0]:
                out[b, j], lse[b, j] = z.softmax(-1) @ keys, z.logsumexp(-1)
    return out, lse


def _weights_exact(s):
    c, got = s["case"], s["weight"].double()
    pos, n = s["q_pos"].tolist(), s["n_entries"].tolist()
    for b in range(c["B"]):
        at = torch.arange(c["N"], device=DEV) if s["idx"] is None else s["idx"][b][s["idx"][b] >= 0].long()
        for j in range(c["nq"]):
            seen = at[at < min((pos[b][j] + 1) // c["m"], n[b])]
            z = s["kv"][b, seen].double() @ s["q"][b, j].double().t() * c["D"] ** -0.5
            got[b].index_add_(0, seen, torch.exp(z - s["lse"][b, j].double()).sum(1))
    return got


def _evict_exact(s):
    c, w, n = s["case"], s["weight"].cpu().numpy().copy(), s["n_entries"].tolist()
    idx, kept = np.full((c["B"], c["budget"]), -1, np.int32), np.zeros(c["B"], np.int32)
    for b in range(c["B"]):
        fit = [i for i in range(n[b]) if w[b, i] >= 0]
        new = [i for i in fit if i >= n[b] - c["recent"]][-c["budget"]:]
        old = sorted((i for i in fit if i < n[b] - c["recent"]), key=lambda i: (-w[b, i], i))[:c["budget"] - len(new)]
        keep = sorted(old + new)
        idx[b, :len(keep)], kept[b] = keep, len(keep)
        w[b, np.setdiff1d(np.arange(n[b]), keep)] = -1
    return idx, kept, w.astype(np.float64)


def exact(case, seed):
    return globals()["_" + case["op"] + "_exact"](prepare(case, seed))
