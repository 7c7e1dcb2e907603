"""Rotary positions, shared-prefix attention, entry weights and eviction on the
GPU, against their definitions in 64 bits (longctx_ref)."""
import math
import threading

import pytest
import torch

import longctx_ref as ref
from long_context_compressed_03_b200 import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, dt, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(dt)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def within(got, want, bound, what):
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: infinities or NaN differ"
    fin = torch.isfinite(want)
    bad = ((got - want).abs() > bound)[fin]
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got - want).abs() - bound)[fin].max()))


# ------------------------------------------------------------------ rotary positions
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,n,H,Hy,D,rot,off", [
    (1, 1, 1, 0, 16, 2, 0), (3, 1, 64, 1, 128, 64, 64), (2, 37, 5, 2, 64, 64, 0), (1, 200, 1, 1, 128, 32, 96),
    (2, 9, 3, 1, 80, 50, 30), (1, 5, 2, 0, 33, 14, 3), (5, 3, 16, 1, 256, 256, 0), (1, 1000, 1, 0, 64, 16, 8)])
def test_rope(dt, interleaved, B, n, H, Hy, D, rot, off):
    g = gen(B * 1000 + n + D)
    x, y = normal(g, dt, B, n, H, D), normal(g, dt, B, n, Hy, D) if Hy else None
    pos = torch.randint(0, 1 << 20, (B, n), generator=g, device=DEV, dtype=torch.int32)
    pos[0, 0] = 0
    pos[-1, -1] = (1 << 31) - 1
    if n > 2:
        pos[-1, n // 2] = -1
    freqs, scale = api.rope_freqs(rot, factor=16.0, original_len=65536)
    for transpose in (False, True):
        out = api.rope(x, freqs, pos=pos, y=y, rot_offset=off, interleaved=interleaved, scale=scale,
                       transpose=transpose)
        for v, o in zip((x, y), out):
            if v is None:
                assert o is None
                continue
            want, bound = ref.rope(v, pos, freqs, off, interleaved, scale, transpose)
            within(o, want, bound, "rope")
        xi, yi = x.clone(), None if y is None else y.clone()
        api.csa_rope(xi, xi, freqs, y=yi, y_out=yi, pos=pos, rot_offset=off, interleaved=interleaved,
                     scale=scale, transpose=transpose)
        assert torch.equal(xi, out[0]) and (y is None or torch.equal(yi, out[1]))


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,n,H,Hy,D,rot,off", [
    # rotated parts that are no whole vectors, in rows that are and are not; many tokens a CTA,
    # one token's rows over several CTAs, rows of more items than a CTA's threads
    (2, 700, 17, 1, 80, 50, 0), (1, 3, 300, 2, 192, 50, 142), (3, 1, 64, 1, 80, 50, 30), (1, 260, 2, 2, 36, 6, 5),
    (1, 4, 3, 1, 1100, 250, 3), (1, 4, 2, 0, 1104, 256, 8), (4, 90, 1, 1, 16, 2, 7), (64, 2, 3, 2, 64, 64, 0)])
def test_rope_of_odd_parts_and_in_place(dt, interleaved, B, n, H, Hy, D, rot, off):
    g = gen(B * 1000 + n + D)
    x, y = normal(g, dt, B, n, H, D), normal(g, dt, B, n, Hy, D) if Hy else None
    pos = torch.randint(-1, 1 << 20, (B, n), generator=g, device=DEV, dtype=torch.int32)
    freqs, _ = api.rope_freqs(rot)
    out = api.rope(x, freqs, pos=pos, y=y, rot_offset=off, interleaved=interleaved)
    for t, o in zip((x, y), out):
        if t is not None:
            want, bound = ref.rope(t, pos, freqs, off, interleaved, 1.0, False)
            within(o, want, bound, "rope")
    api.csa_rope(x, x, freqs, y=y, y_out=y, pos=pos, rot_offset=off, interleaved=interleaved)
    assert torch.equal(x, out[0]) and (y is None or torch.equal(y, out[1]))


@pytest.mark.parametrize("dt,D,extra", [(BF, 128, 1), (F32, 64, 3), (BF, 24, 1)])
def test_rope_strided_views_and_default_positions(dt, D, extra):
    g, B, n, H = gen(3), 2, 17, 6
    fused = normal(g, dt, B, n, H + extra, D)
    x = fused[:, :, :H]
    freqs, _ = api.rope_freqs(D // 2)
    pos = (5 + 4 * torch.arange(n, device=DEV, dtype=torch.int32)).expand(B, n)
    want, bound = ref.rope(x, pos, freqs, 0, False, 1.0, False)
    out, _ = api.rope(x, freqs, pos0=5, pos_step=4, interleaved=False)
    within(out, want, bound, "rope of a view")
    rest = fused[:, :, H:].clone()
    api.csa_rope(x, x, freqs, pos0=5, pos_step=4, interleaved=False)          # in place in the view
    assert torch.equal(x, out) and torch.equal(fused[:, :, H:], rest)
    void = torch.full((B, n), -1, dtype=torch.int32, device=DEV)
    v = normal(g, dt, B, n, H, D)
    v[0, 0, 0, 0] = math.inf
    v[0, 1, 0, 1] = math.nan
    same, _ = api.rope(v, freqs, pos=void)
    assert torch.equal(same.view(torch.uint8), v.view(torch.uint8))           # passed on bit for bit


def test_rope_into_a_view_between_its_input():
    # heads 2 and 3 of a buffer's five receive the rotation of heads 0 and 1
    g, B, n = gen(95), 2, 9
    buf = normal(g, BF, B, n, 5, 64)
    freqs, _ = api.rope_freqs(32)
    rest, want = buf[:, :, 4].clone(), api.rope(buf[:, :, :2], freqs, pos0=3)[0]
    first = buf[:, :, :2].clone()
    api.csa_rope(buf[:, :, :2], buf[:, :, 2:4], freqs, pos0=3)
    assert torch.equal(buf[:, :, 2:4], want) and torch.equal(buf[:, :, :2], first) and torch.equal(buf[:, :, 4], rest)
    for bad in (buf[:, :, 1:3], buf[:, 1:, :2]):           # outputs that share elements with their input
        with pytest.raises((api.CsaError, ValueError)):
            api.csa_rope(buf[:, :bad.shape[1], :2], bad, freqs)


def exact_turns(freq, pos):
    """pos * freq as a fraction of a turn in [-1/2, 1/2), of 1000-bit integers (freq: a float)."""
    one = 1 << 1000

    def atan_inv(n):                                   # one * arctan(1 / n)
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    pi = 4 * (4 * atan_inv(5) - atan_inv(239))         # Machin
    num, den = float(freq).as_integer_ratio()
    turn = pos * num * one * one // (den * 2 * pi) % one
    return (turn - one if 2 * turn >= one else turn) / one


def test_rope_angles_of_large_frequencies_and_far_positions():
    # cos and sin themselves: x = (1, 0) in every pair.  The angle is within 2^-27 of a turn (and
    # 2^-32 where it is less than 2^-8 of a turn from a quarter turn), sincospi within 2 ulp
    freqs = [1.0, 0.1, 3.0, 1234.5, -1234.5, 1e6, -1e6, 999999.125, 1e-3, 2.0 ** -30, 0.0, 6.283185307179586]
    far = [0, 1, 77, 4097, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, (1 << 31) - 1]
    f = torch.tensor(freqs, dtype=torch.float64)
    x = torch.zeros(1, len(far), 1, 2 * len(freqs), device=DEV)
    x[..., 0::2] = 1.0
    got = api.rope(x, f, pos=i32([far]))[0][0, :, 0].double().cpu()
    for t, p in enumerate(far):
        for j, fr in enumerate(freqs):
            turn = exact_turns(fr, p)
            c, s = math.cos(2 * math.pi * turn), math.sin(2 * math.pi * turn)
            for v, w in ((float(got[t, 2 * j]), c), (float(got[t, 2 * j + 1]), s)):
                assert abs(v - w) <= 2 * math.pi * 2.0 ** -27 + 2.0 ** -22 * abs(w), (fr, p, v, w)
    # positions whose angle is close to a quarter, half or three quarters of a turn (freq 0.01)
    near = [p for p in range(200000) if abs((4 * p * 0.01 / (2 * math.pi)) % 1.0 - 0.5) > 0.5 - 2.0 ** -6]
    x = torch.zeros(1, len(near), 1, 2, device=DEV)
    x[..., 0] = 1.0
    got = api.rope(x, torch.tensor([0.01], dtype=torch.float64), pos=i32([near]))[0][0, :, 0].double().cpu()
    # (p * 0.01 in fp64: within 2^-42 rad of the frequency's own product)
    ang = torch.tensor(near, dtype=torch.float64) * 0.01
    want = torch.stack([ang.cos(), ang.sin()], 1)
    assert float(((got - want).abs() - 2.0 ** -22 * want.abs()).max()) <= 2 * math.pi * 2.0 ** -32 + 2.0 ** -42


def test_rope_gradient():
    # the transposed call is the gradient of the rotation: against central differences of
    # sum(w * rope(x)), which is linear in x, so a difference over any step is exact up to rounding
    g, B, n, H, D = gen(8), 1, 4, 2, 16
    x, w = normal(g, F32, B, n, H, D), normal(g, F32, B, n, H, D)
    pos = i32([[3, 70000, 12, 999999]])
    freqs, scale = api.rope_freqs(8, factor=4.0, original_len=4096)
    kw = dict(pos=pos, rot_offset=4, scale=scale)
    grad, _ = api.rope(w, freqs, transpose=True, **kw)
    for k in range(0, x.numel(), 7):
        e = torch.zeros_like(x)
        e.view(-1)[k] = 1.0
        hi, lo = api.rope(x + e, freqs, **kw)[0].double(), api.rope(x - e, freqs, **kw)[0].double()
        diff = float((w.double() * (hi - lo)).sum()) / 2
        # each of the four rotated values carries 4.6e-7 of |a| + |b| (<= 12 here) and of scale
        # (1.14), times |w| <= 4, and x +- 1 rounds once
        assert abs(diff - float(grad.view(-1)[k])) <= 4 * 4 * (4.6e-7 * 12 * 1.14 + 2.0 ** -22)
    back, _ = api.rope(api.rope(x, freqs, pos=pos)[0], freqs, pos=pos, transpose=True)
    assert float((back - x).abs().max()) <= 2 * 2 * 4.6e-7 * 12           # scale 1: the inverse


def test_rope_from_several_host_threads():
    # calls whose CTAs need different amounts of shared memory, at the same time
    lib, calls = api.load(), []
    for k, (shape, rot) in enumerate((((1, 32768, 1, 128), 64), ((64, 1, 65, 128), 64), ((1, 9000, 1, 80), 50),
                                      ((3, 1, 17, 80), 50))):
        B, n, H, D = shape
        x, freqs = normal(gen(91 + k), BF, *shape), api.rope_freqs(rot)[0]
        out, s = torch.empty_like(x), torch.cuda.Stream()
        args = (x.data_ptr(), out.data_ptr(), H, None, None, None, 0, None, api.DT_BF16, B, n, D, rot, 0, 0,
                freqs.data_ptr(), 1.0, None, 0, 1, 0, s.cuda_stream)
        calls.append((args, x, freqs, out, s, api.rope(x, freqs, interleaved=False)[0]))
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(calls)), [0] * len(calls)

    def work(k):
        args, f = calls[k][0], lib.csa_rope
        start.wait()
        for _ in range(20000):
            failed[k] += f(*args) != api.CSA_OK

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(calls)
    assert all(torch.equal(c[3], c[5]) for c in calls)


# ------------------------------------------------------------------ shared prefix
def prefix_case(seed, dt, B, nq, H, D, Np, cap, W, m=4, L=None, void=()):
    g = gen(seed)
    L = W + nq - 1 if L is None else L
    own = torch.randint(0, cap + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    last = (Np + own) * m + torch.randint(0, m, (B,), generator=g, device=DEV, dtype=torch.int32) - 1 + nq * m
    pos = last[:, None] - (nq - 1) + torch.arange(nq, device=DEV, dtype=torch.int32)
    for b in void:
        pos[b] = -1
    return dict(q=normal(g, dt, B, nq, H, D), kv_p=normal(g, dt, Np, D), kv_c=normal(g, dt, B, cap, D), m=m,
                kv_raw=normal(g, dt, B, L, D), window=W, n_entries=(Np + own).contiguous(),
                raw_pos0=(last - (L - 1)).contiguous(), raw_len=i32([L] * B), q_pos=pos.contiguous())


def run_prefix(a, **kw):
    a = dict(a)
    return api.hca_attn_prefix(a.pop("q"), a.pop("kv_p"), a.pop("kv_c"), a.pop("m"), a.pop("kv_raw"),
                               a.pop("window"), with_lse=True, **a, **kw)


def check_prefix(a, dt, **kw):
    out, lse = run_prefix(a, **kw)
    want, wl, bound, bl = ref.prefix_attention(dict(a, scale=kw.get("softmax_scale")), dt, BF if dt == BF else None)
    within(out, want, bound, "prefix attention")
    within(lse, wl, bl, "prefix attention lse")
    return out, lse


@pytest.mark.parametrize("dt,B,nq,H,D,Np,cap,W", [
    (BF, 1, 1, 64, 128, 1, 0, 0), (BF, 1, 1, 64, 128, 128, 0, 1), (BF, 3, 1, 64, 128, 129, 3, 16),
    (BF, 2, 2, 64, 128, 700, 70, 65), (BF, 5, 3, 64, 128, 383, 200, 130), (BF, 4, 1, 128, 128, 260, 9, 40),
    (BF, 3, 2, 128, 128, 511, 129, 128), (BF, 9, 1, 64, 128, 1000, 1, 300), (BF, 3, 1, 16, 64, 90, 10, 20),
    (BF, 3, 1, 32, 128, 300, 10, 20), (BF, 2, 1, 64, 128, 0, 40, 20), (BF, 2, 2, 64, 128, 0, 0, 33),
    (F32, 2, 3, 8, 64, 300, 20, 32), (F32, 1, 1, 8, 64, 1, 0, 0), (F32, 3, 1, 16, 128, 77, 5, 9),
    (F32, 2, 1, 64, 128, 130, 5, 9), (F32, 5, 1, 8, 64, 1000, 40, 100)])
def test_prefix_attention(dt, B, nq, H, D, Np, cap, W):
    check_prefix(prefix_case(B * 100 + Np, dt, B, nq, H, D, Np, cap, W), dt)


@pytest.mark.parametrize("dt,B,nq,H,D,Np,cap,W", [
    # each head count and width; rows that share clusters of 8, 4 and 2 CTAs, and rows alone
    (BF, 2, 1, 16, 128, 4000, 30, 100), (BF, 1, 3, 32, 64, 2500, 7, 60), (BF, 2, 2, 64, 64, 1500, 33, 70),
    (BF, 1, 2, 128, 64, 900, 10, 128), (BF, 2, 1, 8, 128, 1111, 5, 17), (BF, 2, 2, 8, 64, 64, 0, 0),
    (BF, 40, 1, 8, 64, 130, 9, 33), (BF, 75, 2, 16, 64, 200, 9, 33), (BF, 150, 1, 8, 128, 70, 3, 8),
    (BF, 4, 1, 32, 128, 0, 70, 20), (BF, 1, 1, 16, 128, 17000, 0, 0), (BF, 1, 1, 32, 128, 1, 0, 0),
    (F32, 37, 1, 8, 64, 90, 30, 20), (F32, 74, 1, 16, 64, 65, 3, 8), (F32, 75, 2, 8, 64, 40, 3, 8),
    (F32, 1, 1, 128, 128, 333, 5, 9), (F32, 1, 2, 32, 128, 0, 300, 5), (F32, 1, 1, 8, 128, 255, 0, 1)])
def test_prefix_attention_of_other_heads(dt, B, nq, H, D, Np, cap, W):
    check_prefix(prefix_case(B * 100 + Np + H, dt, B, nq, H, D, Np, cap, W, void=(B // 2,) if B > 2 else ()), dt)


@pytest.mark.parametrize("H", [64, 128])
@pytest.mark.parametrize("where", ["first tile", "shared", "own", "window"])
@pytest.mark.parametrize("gap", [30.0, 80.0, 500.0])
def test_prefix_score_far_above_the_first_ones(H, where, gap):
    # one key whose score is `gap` powers of two above all others, the first key's among them:
    # weights of 2^gap against it fit an fp32 sum, pass 2^64, or overflow
    a = prefix_case(51, BF, 3, 2, H, 128, 900, 60, 100, m=4)
    u = (torch.randint(0, 2, (128,), generator=gen(52), device=DEV) * 2 - 1).to(BF)
    sign = torch.ones(H, 1, device=DEV, dtype=BF)
    sign[1::2] = -1                                        # (every other head sees it far below)
    a["q"] = (u * sign).expand_as(a["q"]).contiguous()
    c = gap * math.log(2.0) / math.sqrt(128.0)             # u . (c u) / sqrt(128) = gap ln 2
    far = (u.float() * c).to(BF)
    a["n_entries"] = i32([960, 960, 950])
    a["q_pos"] = i32([[3898, 3899]] * 3)
    a["raw_pos0"] = i32([3899 - a["kv_raw"].shape[1] + 1] * 3)
    for k in ("kv_p", "kv_c", "kv_raw"):
        a[k] = a[k] * 0.25
    if where == "first tile":
        a["kv_p"][77] = far
    elif where == "shared":
        a["kv_p"][500] = far
    elif where == "own":
        a["kv_c"][1, 45] = far
    else:
        a["kv_raw"][2, 70] = far
    check_prefix(a, BF)


@pytest.mark.parametrize("dt,H,D", [(BF, 64, 128), (BF, 128, 128), (BF, 16, 64), (BF, 32, 128), (BF, 8, 128),
                                    (F32, 8, 64)])
def test_prefix_partial_visibility_empty_rows_and_poison(dt, H, D):
    # rows that see no key, only part of the prefix, no window, a cache slot before position 0;
    # whatever a row may not see is NaN or infinite
    B, nq, Np, cap, W, m, L = 7, 2, 300, 50, 24, 4, 40
    a = prefix_case(5, dt, B, nq, H, D, Np, cap, W, m=m, L=L)
    a["n_entries"] = i32([0, 10, 130, 299, 300, 301, 345])
    a["q_pos"] = i32([[-1, 2], [5, 4000], [-1, -1], [1100, 1201], [5000, 5001], [1203, 1204], [9000, 9001]])
    a["raw_pos0"] = i32([-30, -8, 0, 1170, 4970, 1180, 8000])
    a["raw_len"] = i32([40, 20, 0, 40, 32, 25, 40])
    vis = torch.minimum((a["q_pos"] + 1) // m, a["n_entries"][:, None]).amax(1)
    for b in range(B):
        own = max(int(vis[b]) - Np, 0)
        a["kv_c"][b, own:] = math.nan if b % 2 else math.inf
        for i in range(L):
            p = int(a["raw_pos0"][b]) + i
            if i >= int(a["raw_len"][b]) or p < 0 or p > int(a["q_pos"][b].max()):
                a["kv_raw"][b, i] = -math.inf if b % 2 else math.nan
    out, lse = check_prefix(a, dt)
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())
    # a prefix poisoned past what a group of elements sees leaves those elements finite
    a["kv_p"][130:] = math.nan
    out, lse = run_prefix(a)
    want, wl, bound, bl = ref.prefix_attention(a, dt, BF if dt == BF else None)
    for b in range(3):
        within(out[b], want[b], bound[b], "below the poison")
        within(lse[b], wl[b], bl[b], "below the poison")
    a["n_entries"] = a["n_entries"].clamp(max=130)
    a["kv_c"][:] = math.nan
    check_prefix(a, dt)


@pytest.mark.parametrize("nq", [1, 2])
@pytest.mark.parametrize("where", ["own", "window", "rest of the prefix"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_prefix_non_finite_keys_stay_with_the_rows_that_see_them(where, value, nq):
    # 64 heads: two rows share the MMA's 128 lanes and an own tile holds 64 keys of each.  One key
    # of one of the two is not finite; the row that does not see it keeps its result
    B, Np, cap, W, m = 4, 300, 90, 100, 4
    a = prefix_case(81 + nq, BF, B, nq, 64, 128, Np, cap, W, m=m)
    a["n_entries"], last = i32([Np + 70, Np + 80, Np + 75, Np + 90]), i32([1490, 1507, 1499, 1567])
    if where == "rest of the prefix":                # only row (0, 0) sees less than the whole prefix
        a["n_entries"][0] = 140
    a["q_pos"] = (last[:, None] - (nq - 1) * m + m * torch.arange(nq, device=DEV, dtype=torch.int32)).contiguous()
    a["raw_pos0"] = (last - (a["kv_raw"].shape[1] - 1)).contiguous()
    bad = [(1, j) for j in range(nq)]                # (the unit's other row: (0, 0), or for two rows an element (1, 0))
    if where == "own":
        vis = int((a["q_pos"][1, -1] + 1) // m)      # the entry that only element 1's last row sees
        a["kv_c"][1, (min(vis, Np + 80) - Np - 1) if nq == 2 else 33] = value
        bad = bad[-1:]
    elif where == "window":
        a["kv_raw"][1, -1 if nq == 2 else 7] = value
        bad = bad[-1:]
    else:
        a["kv_p"][150] = value                       # (in a tile that has keys of both)
        bad = [(b, j) for b in range(1, B) for j in range(nq)]
    out, lse = run_prefix(a)
    want, wl, bound, bl = ref.prefix_attention(a, BF, BF)
    for b in range(B):
        for j in range(nq):
            if (b, j) in bad:
                assert not bool(torch.isfinite(out[b, j].float()).any())
                continue
            assert bool(torch.isfinite(want[b, j]).all())
            within(out[b, j], want[b, j], bound[b, j], f"row {b}, {j}")
            within(lse[b, j], wl[b, j], bl[b, j], f"lse of row {b}, {j}")


@pytest.mark.parametrize("dt,H,D", [(F32, 8, 64), (F32, 64, 128), (BF, 8, 128)])
def test_prefix_a_visible_nan_is_not_an_empty_row(dt, H, D):
    # clusters of CTAs a row: the key is one CTA's, the others' keys are finite
    a = prefix_case(88, dt, 2, 1, H, D, 400, 20, 64)
    a["kv_c"][1, 0] = math.nan
    a["n_entries"], a["q_pos"] = i32([410, 410]), i32([[1700], [1700]])
    a["raw_pos0"] = i32([1637, 1637])
    out, lse = run_prefix(a)
    want, wl, bound, bl = ref.prefix_attention(a, dt, BF if dt == BF else None)
    within(out[0], want[0], bound[0], "the other element")
    within(lse[0], wl[0], bl[0], "its lse")
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())


def test_attention_from_several_host_threads():
    # the cluster-split kernel's shared memory goes with the keys a CTA has
    lib, calls = api.load(), []
    for k, (B, Np, cap) in enumerate(((2, 30, 5), (60, 9000, 9), (1, 700, 20), (111, 2000, 3))):
        a = prefix_case(141 + k, BF, B, 1, 16, 64, Np, cap, 8)
        out, s = torch.empty_like(a["q"]), torch.cuda.Stream()
        ptr = {n: a[n].data_ptr() for n in ("q", "kv_p", "kv_c", "n_entries", "kv_raw", "raw_pos0", "raw_len", "q_pos")}
        args = (ptr["q"], api.DT_BF16, B, 1, 16, 64, ptr["kv_p"], Np, ptr["kv_c"], cap, ptr["n_entries"], 4, ptr["kv_raw"],
                8, ptr["raw_pos0"], ptr["raw_len"], 8, ptr["q_pos"], 0.0, out.data_ptr(), None, None, 0, s.cuda_stream)
        calls.append((args, a, out, s, run_prefix(a)[0]))
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(calls)), [0] * len(calls)

    def work(k):
        args, f = calls[k][0], lib.hca_dense_attn_prefix
        start.wait()
        for _ in range(4000):
            failed[k] += f(*args) != api.CSA_OK

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(calls)
    assert all(torch.equal(c[2], c[4]) for c in calls)


@pytest.mark.parametrize("H,B", [(64, 1), (64, 2), (128, 1), (128, 30)])
@pytest.mark.parametrize("value", [math.nan, -math.inf])
def test_prefix_a_part_of_nothing_but_nan(H, B, value):
    # the last key, alone in its tile, gives every score NaN; cut units leave it a part of its own
    a = prefix_case(89, BF, B, 1, H, 128, 385, 0, 0)
    a["n_entries"], a["q_pos"] = i32([385] * B), i32([[4 * 385]] * B)
    a["kv_p"][384] = value
    out, lse = run_prefix(a)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    a["n_entries"][0] = 384                                # element 0 does not see it
    out, lse = run_prefix(a)
    want, wl, bound, bl = ref.prefix_attention(a, BF, BF)
    within(out[0], want[0], bound[0], "element 0")
    within(lse[0], wl[0], bl[0], "lse of element 0")
    assert bool(torch.isnan(out[1:]).all()) and bool(torch.isnan(lse[1:]).all())


@pytest.mark.parametrize("H", [64, 128])
def test_prefix_defaults_scale_and_large_scores(H):
    # no optional arrays (positions 0 .. n_q - 1: a prefill over a prefix of m = 1 entries), a given
    # scale, keys of magnitude ~50 (one weight close to 1)
    g = gen(11)
    a = dict(q=normal(g, BF, 2, 130, H, 128), kv_p=normal(g, BF, 70, 128) * 4, kv_c=normal(g, BF, 2, 30, 128),
             m=1, kv_raw=normal(g, BF, 2, 130, 128), window=20, n_entries=None, raw_pos0=None, raw_len=None,
             q_pos=None)
    check_prefix(a, BF, softmax_scale=0.5)


@pytest.mark.parametrize("H,nq", [(64, 1), (128, 1), (64, 2)])
@pytest.mark.parametrize("Np", [100, 700])
def test_prefix_first_key_of_the_lowest_value(H, nq, Np):
    # the first key's score is below fp32's range (a masked entry of the type's lowest value), all
    # the others' are 2^-196 in weight against a score of 0
    a = prefix_case(98, BF, 3, nq, H, 128, Np, 20, 30)
    a["n_entries"], a["q_pos"] = i32([Np + 20, Np + 7, Np]), (i32([[4 * Np + 100 + j for j in range(nq)]] * 3)).contiguous()
    a["raw_pos0"] = (a["q_pos"][:, -1] - (a["kv_raw"].shape[1] - 1)).contiguous()
    a["q"] = a["q"] * 0.125
    for k in ("kv_p", "kv_c", "kv_raw"):
        a[k] = a[k] * 0.125
        a[k][..., 5:7] = torch.tensor([0.0, -48.0], device=DEV, dtype=BF)
    a["q"][..., 5:7] = torch.tensor([4.0, 32.0], device=DEV, dtype=BF)
    a["kv_p"][0] = 0.0
    a["kv_p"][0, 5] = -3e38
    a["kv_raw"][1, 0] = a["kv_p"][0]                       # (own tiles begin with the window)
    check_prefix(a, BF)


def test_prefix_matches_dense_call_on_the_whole_cache():
    a = prefix_case(21, BF, 6, 1, 64, 128, 900, 60, 128, m=128)
    out, lse = run_prefix(a)
    whole = torch.cat([a["kv_p"].expand(6, -1, -1), a["kv_c"]], 1).contiguous()
    o2, l2 = api.hca_attn(a["q"], whole, 128, a["kv_raw"], 128, with_lse=True, n_entries=a["n_entries"],
                          raw_pos0=a["raw_pos0"], raw_len=a["raw_len"], q_pos=a["q_pos"])
    want, wl, bound, bl = ref.prefix_attention(a, BF, BF)
    assert bool(((out.double() - o2.double()).abs() <= 2 * bound).all())
    assert bool(((lse.double() - l2.double()).abs() <= 2 * bl).all())


def test_prefix_is_deterministic_and_leaves_its_inputs():
    a = prefix_case(31, BF, 33, 1, 64, 128, 1500, 40, 200, m=128)
    before = {k: v.clone() for k, v in a.items() if isinstance(v, torch.Tensor)}
    o1, l1 = run_prefix(a)
    for _ in range(3):
        o2, l2 = run_prefix(a)
        assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert all(torch.equal(a[k], v) for k, v in before.items())


# ------------------------------------------------------------------ entry weights
def weights_case(seed, dt, B, nq, H, D, N, m=4, topk=0):
    g = gen(seed)
    q, kv = normal(g, dt, B, nq, H, D), normal(g, dt, B, N, D)
    ne = torch.randint(N // 2, N + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    pos = ((ne * m + m - 2)[:, None] - (nq - 1) + torch.arange(nq, device=DEV, dtype=torch.int32)).contiguous()
    lse = torch.rand(B, nq, H, generator=g, device=DEV) + math.log(N + 1)
    idx = None
    if topk:
        idx = torch.rand(B, N, generator=g, device=DEV).argsort(1)[:, :topk].to(torch.int32).contiguous()
    return dict(q=q, kv=kv, m=m, lse=lse, weight=torch.rand(B, N, generator=g, device=DEV), idx=idx, n_entries=ne,
                q_pos=pos)


def run_weights(a, **kw):
    a = dict(a)
    return api.entry_weights(a.pop("q"), a.pop("kv"), a.pop("m"), a.pop("lse"), **a, **kw)


def check_weights(a):
    got = run_weights(a)
    want, bound = ref.entry_weights(a["q"], a["kv"], a["m"], a["lse"], a["weight"], a["idx"], a["n_entries"], a["q_pos"])
    within(got, want, bound, "entry weights")
    return got


@pytest.mark.parametrize("dt,B,nq,H,D,N,topk", [
    (BF, 1, 1, 64, 128, 1, 0), (BF, 3, 1, 64, 128, 130, 0), (BF, 2, 1, 128, 128, 700, 0), (BF, 2, 5, 64, 128, 259, 0),
    (BF, 1, 3, 16, 64, 500, 0), (BF, 2, 1, 8, 128, 77, 0), (BF, 2, 2, 5, 48, 33, 0), (BF, 3, 1, 64, 128, 600, 77),
    (BF, 1, 33, 64, 128, 1030, 0), (BF, 2, 3, 64, 128, 300, 130), (BF, 1, 70, 2, 128, 140, 0),
    (F32, 2, 1, 8, 64, 300, 0), (F32, 2, 3, 8, 64, 65, 10), (F32, 1, 1, 64, 256, 40, 0)])
def test_entry_weights(dt, B, nq, H, D, N, topk):
    check_weights(weights_case(B * 10 + N, dt, B, nq, H, D, N, topk=topk))


@pytest.mark.parametrize("dt", [BF, F32])
def test_entry_weights_masks_lists_and_poison(dt):
    a = weights_case(3, dt, 5, 3, 8, 64, 200, m=4)
    a["n_entries"] = i32([0, 1, 100, 250, 200])
    a["q_pos"] = i32([[500, 501, 502], [2, 3, 4], [-1, 300, -1], [700, 798, 799], [-1, -1, -1]])
    a["lse"][2, 1, 3] = -math.inf                       # an empty row adds nothing
    a["lse"][3, 0] = -math.inf
    for b, seen in enumerate((0, 1, 75, 200, 0)):
        a["kv"][b, seen:] = math.nan if b % 2 else math.inf
    got = check_weights(a)
    assert torch.equal(got[0], a["weight"][0]) and torch.equal(got[4], a["weight"][4])
    a["weight"] = None
    check_weights(a)
    # lists: padding, entries outside the cache or not visible, an entry twice
    a["weight"] = torch.rand(5, 200, device=DEV)
    a["idx"] = i32([[0, 5, -1, 7]] * 2 + [[74, 75, 74, -3], [199, 0, 250, 199], [1, 2, 3, 4]])
    check_weights(a)
    w = a["weight"].clone()
    api.hca_entry_weights(a["q"], a["kv"], a["m"], a["lse"], w, weight_in=w, idx=a["idx"], n_entries=a["n_entries"],
                          q_pos=a["q_pos"])             # in place
    assert torch.equal(w, run_weights(a))


@pytest.mark.parametrize("dt,H,D", [(BF, 64, 128), (BF, 16, 64), (F32, 8, 64)])
def test_entry_weights_of_empty_lists_and_no_rows(dt, H, D):
    a = weights_case(73, dt, 3, 2, H, D, 70, m=1)
    none = torch.empty(3, 0, dtype=torch.int32, device=DEV)
    assert torch.equal(run_weights(dict(a, idx=none)), a["weight"])        # an empty list: no entry, not every one
    assert float(run_weights(dict(a, idx=none, weight=None)).abs().max()) == 0
    rows = dict(a, q=a["q"][:, :0], lse=a["lse"][:, :0].contiguous(), q_pos=a["q_pos"][:, :0].contiguous())
    assert torch.equal(run_weights(rows), a["weight"])
    idx, kept = api.evict(a["weight"].clone(), 0)                          # a budget of none, and what follows it
    assert idx.shape == (3, 0) and int(kept.abs().max()) == 0
    assert torch.equal(run_weights(dict(a, idx=idx)), a["weight"])


def test_entry_weights_of_an_attention_call_sum_to_its_heads():
    # with the call's own lse and no window, every head's weights add to one
    g, B, N, H = gen(13), 3, 900, 64
    q, kv = normal(g, BF, B, 1, H, 128), normal(g, BF, B, N, 128)
    pos = i32([[4 * N - 1]] * B)
    _, lse = api.hca_attn(q, kv, 4, torch.zeros(B, 1, 128, dtype=BF, device=DEV), 0, with_lse=True, q_pos=pos)
    w = api.entry_weights(q, kv, 4, lse, q_pos=pos)
    # lse and the scores carry ~1e-5 at most (128 products in fp32), a sum of 900 fp32 terms 900 * 2^-24
    assert float((w.double().sum(1) - H).abs().max()) <= H * 1e-4


# ------------------------------------------------------------------ eviction
@pytest.mark.parametrize("B,N,budget,recent", [
    (1, 1, 1, 0), (1, 1, 0, 0), (3, 33, 7, 2), (2, 1000, 999, 10), (2, 1000, 100, 300), (5, 777, 100, 0),
    (1, 5000, 64, 64), (2, 32768, 2048, 128), (1, 40001, 3001, 1), (3, 2000, 2000, 5), (2, 100, 300, 1000),
    (9, 4096, 512, 17), (1, 150001, 7000, 333)])
def test_evict(B, N, budget, recent):
    g = gen(N + budget)
    w = torch.rand(B, N, generator=g, device=DEV).log().neg()
    w = torch.where(torch.rand(B, N, generator=g, device=DEV) < 0.3, (w * 4).round() / 4, w)     # ties
    w = torch.where(torch.rand(B, N, generator=g, device=DEV) < 0.1, torch.full_like(w, -1), w)
    ne = torch.randint(0, N + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    ne[0] = N
    for n_entries in (ne, None):
        ww = w.clone()
        idx, kept = api.evict(ww, budget, recent=recent, n_entries=n_entries)
        want = ref.evict(w, n_entries, budget, recent)
        assert torch.equal(idx.cpu(), want[0]) and torch.equal(kept.cpu(), want[1]) and torch.equal(ww.cpu(), want[2])
        again = api.evict(ww, budget, recent=recent, n_entries=n_entries)       # nothing more goes
        assert torch.equal(again[0], idx) and torch.equal(again[1], kept)


def test_evict_special_weights():
    w = torch.tensor([[0.0, -0.0, math.nan, math.inf, 1e-45, -1.0, 5.0, 5.0, math.inf, 0.0],
                      [-1.0] * 10, [math.nan] * 10, [0.0] * 10, [7.0] * 10], device=DEV)
    for budget in (0, 1, 2, 3, 4, 5, 6, 8, 10, 12):
        for recent in (0, 1, 3, 20):
            ww = w.clone()
            idx, kept = api.evict(ww, budget, recent=recent)
            want = ref.evict(w, None, budget, recent)
            assert torch.equal(idx.cpu(), want[0]) and torch.equal(kept.cpu(), want[1])
            assert torch.equal(ww.cpu().view(torch.int32), want[2].view(torch.int32))
    ww = w.clone()
    idx, _ = api.evict(ww, 3, n_entries=i32([-5, 3, 99, 4, 0]))      # counts outside the cache are clamped
    want = ref.evict(w, [-5, 3, 99, 4, 0], 3, 0)
    assert torch.equal(idx.cpu(), want[0])


# ------------------------------------------------------------------ together
def test_a_decode_loop_with_eviction():
    """Rotate, append to the compressed cache, attend to the kept entries and the window,
    accumulate the weights, evict -- each step against the definitions."""
    g, B, H, D, m, cap, W, budget, recent = gen(99), 3, 64, 128, 4, 64, 16, 12, 3
    W_c = normal(g, BF, D, D) / math.sqrt(D)
    state = torch.zeros(B, 2, D, device=DEV)
    cache, ne = torch.zeros(B, cap, D, dtype=BF, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    weight, raw = torch.zeros(B, cap, device=DEV), torch.zeros(B, W, D, dtype=BF, device=DEV)
    freqs, _ = api.rope_freqs(64)
    for step in range(90):
        pos = i32([[step]] * B)
        q, kv = api.rope(normal(g, BF, B, 1, H, D), freqs, pos=pos, y=normal(g, BF, B, 1, 1, D), rot_offset=64)
        raw = torch.cat([raw[:, 1:], kv[:, :, 0]], 1).contiguous()
        api.csa_compress_append(kv[:, 0, 0].contiguous(), W_c, m, True, pos[:, 0].contiguous(), state, cache, n_entries=ne)
        before = weight.clone()
        idx, kept = api.evict(weight, budget, recent=recent, n_entries=ne)
        want = ref.evict(before, ne.cpu(), budget, recent)
        assert torch.equal(idx.cpu(), want[0]) and torch.equal(kept.cpu(), want[1])
        p0 = i32([step - W + 1] * B)
        out, lse = api.sparse_attn(q, cache, idx, raw, W, with_lse=True, raw_pos0=p0, raw_len=i32([W] * B), q_pos=pos)
        new = api.entry_weights(q, cache, m, lse, weight=weight, idx=idx, n_entries=ne, q_pos=pos)
        if step % 10 == 9:
            w, bound = ref.entry_weights(q, cache, m, lse, weight, idx, ne, pos)
            within(new, w, bound, "weights")
            for b in range(B):
                keys = torch.cat([cache[b, idx[b][idx[b] >= 0].long()], raw[b, max(0, W - 1 - step):]]).double()
                o, l, bo, bl = ref.attention_row(q[b, 0].double(), keys, D ** -0.5, BF, BF)
                within(out[b, 0], o, bo, "attention over the kept entries")
                within(lse[b, 0], l, bl, "lse over the kept entries")
                assert float(new[b].clamp(min=0).sum()) <= H * (step + 1) * 1.001
        back, _ = api.rope(out, freqs, pos=pos, rot_offset=64, transpose=True)      # shared KV: turn the output back
        assert torch.isfinite(back.float()).all()
        weight = new
    assert int((weight >= 0).sum(1).max()) <= cap and int(kept[0]) == budget


def test_a_shared_prefix_step_with_weights_of_the_own_entries():
    """A step over a shared prefix, then the weights of each element's own entries from the
    call's lse: prefix, own entries and window together give every head one."""
    a = prefix_case(77, BF, 4, 1, 64, 128, 300, 40, 32, m=4)
    out, lse = run_prefix(a)
    B, cap, Np = 4, 40, 300
    pos_own = (a["q_pos"] - Np * a["m"]).contiguous()          # the own cache counts from the prefix's end
    own = api.entry_weights(a["q"], a["kv_c"], a["m"], lse, n_entries=(a["n_entries"] - Np).contiguous(), q_pos=pos_own)
    pre = api.entry_weights(a["q"], a["kv_p"].expand(B, -1, -1).contiguous(), a["m"], lse, q_pos=a["q_pos"])
    win = api.entry_weights(a["q"], a["kv_raw"], 1, lse, q_pos=i32([[31]] * B))
    total = own.double().sum(1) + pre.double().sum(1) + win.double().sum(1)
    assert float((total - 64).abs().max()) <= 64 * 1e-4


@pytest.mark.parametrize("call", ["hca", "csa"])
def test_decode_attention_directly_behind_the_kernel_that_writes_its_inputs(call):
    # the rotation writes q and the window row in place, the attention follows at once: eagerly and
    # in a graph, with other inputs every time
    g, B, N, W, steps = gen(101), 16, 300, 128, 24
    raw = [normal(g, BF, B, 1, 64, 128) for _ in range(steps)]
    rows = [normal(g, BF, B, 1, 1, 128) for _ in range(steps)]
    kv, win = normal(g, BF, B, N, 128), normal(g, BF, B, W, 128)
    pos, p0 = i32([[4 * N + 50]] * B), i32([4 * N + 50 - W + 1] * B)
    idx = torch.rand(B, 1, N, generator=g, device=DEV).argsort(2)[:, :, :64].to(torch.int32).contiguous()
    freqs, _ = api.rope_freqs(64)
    q, row = torch.empty_like(raw[0]), torch.empty_like(rows[0])

    def attend():
        kw = dict(raw_pos0=p0, q_pos=pos)
        if call == "hca":
            return api.hca_attn(q, kv, 4, win, W, **kw)
        return api.sparse_attn(q, kv, idx, win, W, **kw)

    want = []
    for k in range(steps):
        api.csa_rope(raw[k], q, freqs, y=rows[k], y_out=row, pos=pos)
        win[:, -1:] = row[:, 0]
        torch.cuda.synchronize()
        want.append(attend())
        torch.cuda.synchronize()
    win_y = win[:, -1].view(B, 1, 1, 128)                  # the new row's place in the window

    def step(k):
        api.csa_rope(raw[k], q, freqs, y=rows[k].view(B, 1, 1, 128), y_out=win_y, pos=pos)
        return attend()

    for _ in range(3):
        got = [step(k) for k in range(steps)]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(k) for k in range(steps)]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------ streams and graphs
def _ops(a, w, weight):
    out, lse = run_prefix(a)
    x, _ = api.rope(out, w["freqs"], pos=a["q_pos"], transpose=True)
    new = api.entry_weights(a["q"], w["kv"], 4, lse, weight=weight, q_pos=a["q_pos"])
    idx, kept = api.evict(new, 20, recent=3)
    return out, lse, x, new, idx, kept


def test_side_stream_and_captured_graphs():
    a = prefix_case(41, BF, 5, 1, 64, 128, 700, 33, 100, m=4)
    w = dict(kv=normal(gen(42), BF, 5, 90, 128), freqs=api.rope_freqs(64)[0])
    weight = torch.rand(5, 90, device=DEV)
    want = _ops(a, w, weight)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _ops(a, w, weight)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    b = prefix_case(43, BF, 5, 1, 64, 128, 700, 33, 100, m=4)
    want_b = _ops(b, w, weight)
    graphs = []
    for case in (a, b):                       # two graphs, replayed on two streams at once
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            res = _ops(case, w, weight)
        graphs.append((gr, res))
    s2 = torch.cuda.Stream()
    for _ in range(5):
        for _, res in graphs:
            for r in res:
                r.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(graphs[0][1], want))
        assert all(torch.equal(x, y) for x, y in zip(graphs[1][1], want_b))


def test_positions_at_the_end_of_the_range():
    # t + 1 passes 2^31 - 1: every entry is visible (m = 1)
    last = 2 ** 31 - 1
    for dt, H, D in ((BF, 64, 128), (BF, 16, 64), (F32, 8, 64)):
        a = prefix_case(61, dt, 2, 1, H, D, 200, 10, 0, m=1)
        a["q_pos"], a["n_entries"] = i32([[last], [last - 1]]), i32([210, 205])
        check_prefix(a, dt)
        w = weights_case(62, dt, 2, 1, H, D, 150, m=1)
        w["q_pos"] = i32([[last], [last - 1]])
        check_weights(w)


@pytest.mark.parametrize("B,nq,H", [(310, 1, 64), (157, 2, 128), (9400, 1, 64)])
def test_prefix_with_more_units_than_ctas(B, nq, H):
    # several units a CTA, whole and cut; sampled elements against the definition
    a = prefix_case(63, BF, B, nq, H, 128, 140, 5, 9, m=4, void=(B // 2, B - 1))
    out, lse = run_prefix(a)
    for b in sorted({0, 1, B // 3, B // 2, B // 2 + 1, B - 2, B - 1}):
        one = {k: (v[b:b + 1] if isinstance(v, torch.Tensor) and k != "kv_p" else v) for k, v in a.items()}
        want, wl, bound, bl = ref.prefix_attention(one, BF, BF)
        within(out[b:b + 1], want, bound, f"element {b}")
        within(lse[b:b + 1], wl, bl, f"lse of element {b}")
    o2, l2 = run_prefix(a)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("H,Np", [(128, 128), (128, 300), (64, 128), (64, 384)])
def test_prefix_units_that_follow_one_another_keep_their_offsets(H, Np):
    # several units of one or three tiles a CTA (the two groups of softmax warps take the units'
    # first tiles in turn), the scores of neighbouring rows far apart: a row's LSE and, where a
    # unit is cut, its weight in the join go by the offset of its own unit
    B = 1200
    a = prefix_case(97, BF, B, 1, H, 128, Np, 0, 0)
    a["q_pos"] = torch.full_like(a["q_pos"], 4 * Np + 3)
    step = torch.arange(B, device=DEV) * 37 % 11 - 5
    a["q"] = (a["q"].float() * 2.0 ** step[:, None, None, None]).to(BF)
    a["kv_p"][0] = 1.0                                     # (the key that gives the offsets)
    out, lse = run_prefix(a)
    want, wl, bound, bl = ref.prefix_attention(a, BF, BF)
    for _ in range(20):
        within(out, want, bound, "prefix attention")
        within(lse, wl, bl, "lse")
        out, lse = run_prefix(a)


@pytest.mark.parametrize("B,nq,H", [(4440, 1, 128), (4441, 1, 128), (8881, 1, 64), (3, 3001, 64), (9000, 1, 128)])
def test_prefix_of_more_rows_than_a_wave_takes(B, nq, H):
    # 30 units a CTA at most; one more: two waves of whole units, the last of them empty
    a = prefix_case(99, BF, B, nq, H, 128, 130, 2, 3, m=4, void=(B - 2,))
    out, lse = run_prefix(a)
    for b in sorted({0, 1, B // 2, B - 2, B - 1}):
        j = slice(max(0, nq - 40), nq)
        one = {k: (v[b:b + 1] if isinstance(v, torch.Tensor) and k != "kv_p" else v) for k, v in a.items()}
        one["q"], one["q_pos"] = one["q"][:, j], one["q_pos"][:, j]
        want, wl, bound, bl = ref.prefix_attention(one, BF, BF)
        within(out[b:b + 1, j], want, bound, f"element {b}")
        within(lse[b:b + 1, j], wl, bl, f"lse of element {b}")


def test_offsets_past_32_bits():
    # caches and heads whose last rows lie more than 2^31 elements in
    g, B, N = gen(64), 5, 4_000_000
    kv = torch.zeros(B, N, 128, dtype=BF, device=DEV)
    b = B - 1
    kv[b, :300] = normal(g, BF, 300, 128)
    kv[b, N - 300:] = normal(g, BF, 300, 128)
    q = normal(g, BF, B, 1, 64, 128)
    ne, pos = i32([0] * (B - 1) + [300]), i32([[2 ** 30]] * B)
    raw, p0 = normal(g, BF, B, 4, 128), i32([0] * B)
    a = dict(q=q, kv_p=normal(g, BF, 130, 128), kv_c=kv, m=4, kv_raw=raw, window=0, n_entries=(ne + 130).contiguous(),
             raw_pos0=p0, raw_len=i32([4] * B), q_pos=pos)
    out, lse = run_prefix(a)
    one = dict(a, q=q[b:], kv_c=kv[b:, :300], kv_raw=raw[b:], n_entries=i32([430]), raw_pos0=p0[b:], raw_len=i32([4]),
               q_pos=pos[b:])
    want, wl, bound, bl = ref.prefix_attention(one, BF, BF)
    within(out[b:], want, bound, "last element")
    within(lse[b:], wl, bl, "last element's lse")
    idx = torch.full((B, 300), -1, dtype=torch.int32, device=DEV)
    idx[b] = torch.arange(N - 300, N, device=DEV)
    w = api.entry_weights(q, kv, 1, lse, idx=idx, q_pos=pos)
    ww, bound = ref.entry_weights(q[b:], kv[b:, N - 300:], 1, lse[b:], None, None, None, pos[b:])
    within(w[b:, N - 300:], ww, bound, "last entries' weights")
    assert float(w[:, :N - 300].abs().sum()) == 0
    w = api.entry_weights(q, kv, 1, lse, n_entries=ne, q_pos=pos)
    ww, bound = ref.entry_weights(q[b:], kv[b:, :300], 1, lse[b:], None, None, None, pos[b:])
    within(w[b:, :300], ww, bound, "first entries' weights")
    assert float(w[:b].abs().sum()) == 0 and float(w[b, 300:].abs().sum()) == 0
    del kv, a
    freqs, _ = api.rope_freqs(64)
    big = torch.zeros(1, 70000, 64, 512, dtype=BF, device=DEV)
    big[0, -3:] = normal(g, BF, 3, 64, 512)
    got, _ = api.rope(big, freqs, pos=None, rot_offset=448)
    tail, _ = api.rope(big[:, -3:].contiguous(), freqs, pos=i32([[69997, 69998, 69999]]), rot_offset=448)
    assert torch.equal(got[0, -3:], tail[0])


@pytest.mark.parametrize("B,nq,N,topk", [(1030, 1, 130, 0), (1100, 1, 70, 9), (3, 3, 900, 0), (2, 5, 600, 333)])
def test_entry_weights_many_elements_and_steps(B, nq, N, topk):
    # more elements than their counts are kept for, steps of 128 columns with a half one last
    a = weights_case(65, BF, B, nq, 64, 128, N, topk=topk)
    got = run_weights(a)
    for b in sorted({0, 1, B // 2, B - 2, B - 1}):
        one = {k: (v[b:b + 1] if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
        want, bound = ref.entry_weights(one["q"], one["kv"], a["m"], one["lse"], one["weight"], one["idx"],
                                        one["n_entries"], one["q_pos"])
        within(got[b:b + 1], want, bound, f"element {b}")
    if not topk:
        assert torch.equal(got, run_weights(a))


@pytest.mark.parametrize("B,nq,H,N,fill", [
    # few tiles of many steps (clusters of 8, 4 and 2 CTAs a tile), several rounds of them, caches
    # that hold little and caches that are full, elements without entries
    (1, 40, 64, 700, 1.0), (3, 24, 64, 900, 0.6), (1, 64, 64, 9000, 0.4), (1, 64, 64, 9000, 1.0), (2, 8, 128, 3000, 0.5),
    (7, 16, 64, 1500, 0.3), (1, 5, 64, 129, 1.0), (40, 6, 64, 300, 0.9)])
def test_entry_weights_of_tiles_shared_by_clusters(B, nq, H, N, fill):
    a = weights_case(69 + nq, BF, B, nq, H, 128, N)
    a["n_entries"] = i32([0 if b % 3 == 1 else max(1, int(N * fill) - 5 * b) for b in range(B)])
    a["kv"][:, int(N * fill) + 1:] = math.nan              # nothing sees these
    got = check_weights(a)
    assert torch.equal(got, run_weights(a))
    assert torch.equal(got[:, int(N * fill) + 1:], a["weight"][:, int(N * fill) + 1:])


def test_prefix_workspace():
    a = prefix_case(66, BF, 3, 1, 64, 128, 900, 30, 100, m=4)
    want = run_prefix(a)
    need = api.load().hca_dense_attn_prefix_workspace(api.DT_BF16, 3, 1, 64, 128, 900, 30, 100)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)     # (all NaN as fp32)
    got = run_prefix(a, workspace=ws[:need])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((ws[need:] == 0xFF).all())
    for bad in (ws[:need - 1], ws[1:need + 1]):
        with pytest.raises(api.CsaError):
            run_prefix(a, workspace=bad)
    with pytest.raises(ValueError, match="CUDA"):
        run_prefix(a, workspace=ws.cpu())
    with pytest.raises(ValueError, match="contiguous"):
        run_prefix(a, workspace=ws[::2])


@pytest.mark.parametrize("B,H,Np", [(2, 128, 5000), (70, 64, 700), (201, 64, 1000), (201, 64, 3001), (310, 64, 140),
                                      (301, 128, 300)])
def test_prefix_writes_its_workspace_alone(B, H, Np):
    # uneven and even cuts, no cut (201 rows of few tiles: no bytes), more units than CTAs
    a = prefix_case(140 + B, BF, B, 1, H, 128, Np, 30, 100)
    need = api.load().hca_dense_attn_prefix_workspace(api.DT_BF16, B, 1, H, 128, Np, 30, 100)
    assert (need == 0) == (B == 201 and Np == 1000)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = run_prefix(a, workspace=ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    want, wl, bound, bl = ref.prefix_attention(a, BF, BF)
    within(out, want, bound, "prefix attention")
    within(lse, wl, bl, "lse")


def test_timeouts_are_reported_and_the_next_call_runs_clean():
    lib = api.load()
    a, w = prefix_case(67, BF, 70, 1, 64, 128, 700, 30, 100, m=4), weights_case(68, BF, 3, 2, 64, 128, 500)
    many = weights_case(70, BF, 1, 40, 64, 128, 700)
    for run in (lambda: run_prefix(a)[0], lambda: run_weights(w), lambda: run_weights(many)):
        api.csa_check_device_error()
        want = run()
        torch.cuda.synchronize()
        assert lib.csa_debug_set_wait_limit(2_000_000, 1) == api.CSA_OK       # 2 ms, stall the next launch
        try:
            run()
            with pytest.raises(api.CsaError) as ei:
                api.csa_check_device_error(clear=True)
            assert ei.value.status == api.CSA_ERR_TIMEOUT
        finally:
            assert lib.csa_debug_set_wait_limit(0, 0) == api.CSA_OK
        api.csa_check_device_error()
        assert torch.equal(run(), want)
        torch.cuda.synchronize()
        api.csa_check_device_error()


def test_stream_argument():
    a = prefix_case(51, BF, 2, 1, 64, 128, 300, 10, 50, m=4)
    want = run_prefix(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    torch.cuda.synchronize()
    api.hca_dense_attn_prefix(a["q"], a["kv_p"], a["kv_c"], 4, a["kv_raw"], 50, out, lse_out=lse, stream=s,
                              **{k: a[k] for k in ("n_entries", "raw_pos0", "raw_len", "q_pos")})
    s.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
