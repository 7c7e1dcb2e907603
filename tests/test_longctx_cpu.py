"""Host-side checks of the rotary, shared-prefix, entry-weight and eviction entry
points: what they refuse before anything reaches the GPU, and the frequency rule.
CPU only: every call fails validation, is a no-op, or runs on the host."""
import ctypes
import glob
import math
import os
import re

import pytest
import torch

import longctx_ref as ref
from long_context_compressed_03_b200 import api, build as build_mod

FAKE, ODD, ODD4 = (ctypes.c_void_p(v) for v in (0x10000, 0x10001, 0x10004))
INV, UNS, MIS, OK = api.CSA_ERR_INVALID_ARG, api.CSA_ERR_UNSUPPORTED, api.CSA_ERR_MISALIGNED, api.CSA_OK


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return api.load()


def changed(args, **at):
    a = list(args)
    for k, v in at.items():
        a[int(k[1:])] = v
    return a


def st(*v):
    return (ctypes.c_longlong * 4)(*v)


def test_rope_validation(lib):
    f = (ctypes.c_double * 32)(*([0.5] * 32))
    #       x  out   H  xs    y     yo    Hy ys    dt B  n  D   rot off il freqs s   pos  p0 st tr stream
    ok = [FAKE, FAKE, 2, None, None, None, 0, None, 1, 1, 4, 64, 32, 32, 1, f, 1.0, FAKE, 0, 1, 0, None]
    call = lib.csa_rope
    for change, status in [
            (dict(_8=2), INV), (dict(_8=9), INV), (dict(_9=-1), INV), (dict(_2=-1), INV), (dict(_12=31), INV),
            (dict(_12=0), INV), (dict(_13=33), INV), (dict(_13=-1), INV), (dict(_14=2), INV), (dict(_20=3), INV),
            (dict(_15=None), INV), (dict(_16=math.inf), INV), (dict(_16=math.nan), INV), (dict(_0=None), INV),
            (dict(_1=None), INV), (dict(_17=None, _18=-1), INV), (dict(_17=None, _19=-1), INV), (dict(_0=ODD4), MIS),
            (dict(_1=ODD), MIS), (dict(_17=ODD), MIS), (dict(_11=4097), UNS), (dict(_2=4097), UNS),
            (dict(_11=300, _12=258, _13=0), UNS), (dict(_9=1 << 20, _10=1 << 20), UNS),
            (dict(_3=st(128, 64, 128, 32)), INV),          # output heads overlap
            (dict(_3=st(128, 64, 127, 64)), INV),          # output tokens overlap
            (dict(_3=st(128, -64, 128, 64)), INV),
            (dict(_3=st(256, 64, 128, 64)), INV),          # in place with other strides
            (dict(_6=1), INV),                             # a second tensor without its pointers
    ]:
        assert call(*changed(ok, **change)) == status, change
        assert lib.csa_last_error_detail().decode() != ""
    for bad in (math.nan, math.inf, 1e7):
        g = (ctypes.c_double * 32)(*([bad] * 32))
        assert call(*changed(ok, _15=g)) == INV
    for change in (dict(_9=0), dict(_10=0), dict(_2=0)):
        assert call(*changed(ok, **change)) == OK, change


def test_rope_refuses_tensors_that_overlap(lib):
    f = (ctypes.c_double * 32)(*([0.5] * 32))
    p = lambda v: ctypes.c_void_p(0x100000 + v)  # noqa: E731
    one = 4 * 2 * 64 * 2                                   # bytes of [1, 4, 2, 64] bf16
    far = p(1 << 20)

    def call(x, xo, y, yo, xs=None, ys=None, n=4):
        return lib.csa_rope(x, xo, 2, xs, y, yo, 2, ys, 1, 1, n, 64, 32, 0, 1, f, 1.0, None, 0, 1, 0, None)

    def launched(*a, **kw):                                # accepted: it gets as far as the launch
        assert lib.csa_debug_inject_launch_error(719) == OK
        return call(*a, **kw) == api.CSA_ERR_CUDA

    assert call(p(0), p(one // 2), p(8 * one), p(9 * one)) == INV      # x's output inside x
    assert call(p(0), p(one), p(0), p(one)) == INV                     # one output for both
    assert call(p(0), p(0), p(0), p(0)) == INV                         # the same tensor twice, in place
    assert call(p(0), p(one), p(one), p(2 * one)) == INV               # x's output is y
    assert call(p(0), p(one), p(4 * one), p(0)) == INV                 # y's output is x
    assert launched(p(0), p(one), p(0), p(2 * one))                    # one input, two outputs
    assert launched(p(0), p(0), p(one), p(one))                        # neighbours, in place
    # heads 0-1 and 2-3 of one [1, 4, 5, 64] buffer, in place; heads 1-2 overlap the first
    fused = st(320, 64, 320, 64)
    assert launched(p(0), p(0), p(256), p(256), fused, fused)
    assert call(p(0), p(0), p(128), p(128), fused, fused) == INV
    assert call(p(0), p(0), p(256), p(256), fused, st(256, 64, 256, 64)) == INV      # other token strides
    assert launched(p(0), far, p(256), p(2 << 20), st(320, 64, 128, 64), st(320, 64, 128, 64))
    assert call(p(0), p(0), p(128), p(128), fused, fused, n=1) == INV
    assert launched(p(0), p(0), p(256), p(256), fused, fused, n=1)


def test_rope_strides_of_views_that_interleave():
    # (the memory between a view's heads may be the other view's: no refusal of its own here)
    buf = torch.zeros(2, 9, 5, 64)
    assert list(api._rope_strides(buf[:, :, :2], buf[:, :, 2:4], "x")) == [320, 64, 320, 64]
    assert list(api._rope_strides(buf[:, :, :1], torch.zeros(2, 9, 1, 64), "x")) == [320, 64, 64, 64]
    with pytest.raises(ValueError, match="n tokens apart"):
        api._rope_strides(buf[:, 1:], buf[:, 1:], "x")


def test_binding_refuses_other_devices(monkeypatch):
    class Other:                                           # a tensor of device 1, as the binding sees it
        is_cuda, device, dtype, shape = True, "cuda:1", torch.float32, torch.Size((2, 4))

        def get_device(self):
            return 1

    monkeypatch.setattr(api, "_device", lambda: 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        api._same_device(Other())
    with pytest.raises(ValueError, match="on cuda:1, the first tensor on cuda:0"):
        api._shape(Other(), (2, 4), "idx", 0)
    with pytest.raises(ValueError, match="on cuda:1, the first tensor on the host"):
        api._shape(Other(), (2, 4), "idx", -1)
    with pytest.raises(ValueError, match="CUDA tensors"):
        api._shape(torch.zeros(2, 4), (2, 4), "idx", 0)
    with pytest.raises(ValueError, match="CUDA tensors"):
        api._rope_tensor(torch.zeros(1, 2, 1, 8), torch.zeros(1, 2, 1, 8), 1, 2, 8, torch.float32, "y", 0)


def test_rope_freqs(lib):
    f, s = api.rope_freqs(64)
    assert s == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-14, atol=0)
    # the YaRN rule by hand, d_rot 64, base 10^4, original 4096: pair(32) = 64 ln(4096 / (2 pi 32)) / (2 ln 10^4)
    # = 10.47.. -> 10, pair(1) = 22.5.. -> 23
    g, s = api.rope_freqs(64, factor=40.0, original_len=4096)
    assert abs(s - (0.1 * math.log(40.0) + 1)) < 1e-6
    for j in range(32):
        ramp = min(max((j - 10) / 13, 0.0), 1.0)
        assert abs(float(g[j]) - float(f[j]) * (ramp / 40 + 1 - ramp)) <= 1e-14 * float(f[j])
    assert torch.equal(g[:11], f[:11]) and torch.allclose(g[23:], f[23:] / 40, rtol=1e-14, atol=0)
    # a range too short for a ramp still gives finite, falling frequencies
    h, _ = api.rope_freqs(4, factor=2.0, original_len=1)
    assert torch.isfinite(h).all() and h[0] > h[1]
    for kw in (dict(d_rot=0), dict(d_rot=7), dict(d_rot=-2), dict(base=1.0), dict(base=math.nan), dict(factor=0.5),
               dict(factor=math.inf), dict(factor=2.0), dict(factor=2.0, original_len=64, beta_fast=1.0),
               dict(factor=2.0, original_len=64, beta_slow=0.0)):
        with pytest.raises(api.CsaError):
            api.rope_freqs(**{"d_rot": 64, **kw})


def test_rope_binding_refusals(lib):
    x, f = torch.zeros(1, 2, 3, 8), torch.zeros(2, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        api.rope(x, f)
    with pytest.raises(ValueError, match="freqs"):
        api.rope(x, f.float())
    with pytest.raises(ValueError, match="B, n, heads, D"):
        api.rope(x[0], f)
    with pytest.raises(ValueError, match="shape and dtype"):
        api._rope_tensor(torch.zeros(1, 3, 1, 8), torch.zeros(1, 3, 1, 8), 1, 2, 8, x.dtype, "y")
    with pytest.raises(ValueError, match="shape and dtype"):
        api.csa_rope(x, torch.zeros(1, 2, 3, 7), f)


def test_prefix_validation(lib):
    #       q    dt B  nq H   D    kvp   Np   kvc   cap  ne    m  raw   L   p0    len   W   pos   scale out  lse
    ok = [FAKE, 1, 2, 1, 64, 128, FAKE, 100, FAKE, 10, None, 4, FAKE, 16, None, None, 16, None, 0.0, FAKE, None,
          FAKE, 1 << 40, None]
    call = lib.hca_dense_attn_prefix
    for change, status in [
            (dict(_11=0), INV), (dict(_7=-1), INV), (dict(_9=-1), INV), (dict(_7=1 << 30), INV), (dict(_6=None), INV),
            (dict(_8=None), INV), (dict(_12=None), INV), (dict(_0=None), INV), (dict(_19=None), INV), (dict(_1=2), UNS),
            (dict(_1=7), INV), (dict(_5=100), UNS), (dict(_6=ODD4), MIS), (dict(_0=ODD), MIS), (dict(_19=ODD4), MIS),
            (dict(_20=ODD), MIS), (dict(_17=ODD), MIS), (dict(_16=-1), INV), (dict(_2=-1), INV), (dict(_21=ODD4), MIS)]:
        assert call(*changed(ok, **change)) == status, change
    assert call(*changed(ok, _2=0)) == OK and call(*changed(ok, _3=0)) == OK
    assert call(*changed(ok, _1=0, _4=7, _21=None, _22=0)) == UNS      # no kernel for 7 heads
    need = lib.hca_dense_attn_prefix_workspace(1, 2, 1, 64, 128, 100, 10, 16)
    if need:
        assert call(*changed(ok, _22=need - 1)) == INV and "workspace" in lib.csa_last_error_detail().decode()
        assert call(*changed(ok, _21=None)) == INV
    assert lib.hca_dense_attn_prefix_workspace(1, 0, 1, 64, 128, 100, 10, 16) == 0
    assert lib.hca_dense_attn_prefix_workspace(1, 2, 1, 64, 128, -1, 10, 16) == 0


def test_prefix_workspace_goes_with_the_cuts(lib):
    # a CTA leaves two cut parts at most: a prompt of many query rows needs no more than its CTAs do
    size = lambda B, n_q, H: lib.hca_dense_attn_prefix_workspace(1, B, n_q, H, 128, 4096, 100, 128)  # noqa: E731
    part = (128 * 128 + 3 * 128) * 4
    assert 0 < size(1, 1, 64) <= 148 * part
    for B, n_q, H in ((67, 3, 64), (2, 1000, 64), (2, 8192, 64), (4, 2048, 128), (1, 16383, 64)):
        assert size(B, n_q, H) <= 2 * 148 * part, (B, n_q, H)
    assert size(67, 3, 64) > 0 and size(2, 8192, 64) == 0  # (many rows: whole units a CTA, nothing to join)


def test_weights_and_evict_validation(lib):
    #       q    dt B  nq H   D    kv    N   idx   k  ne    m  pos   s    lse   in    out   stream
    ok = [FAKE, 1, 2, 1, 64, 128, FAKE, 50, FAKE, 5, None, 4, None, 0.0, FAKE, None, FAKE, None]
    call = lib.hca_entry_weights
    for change, status in [
            (dict(_1=3), UNS), (dict(_1=-1), INV), (dict(_2=-1), INV), (dict(_9=-1), INV), (dict(_11=0), INV), (dict(_4=0), INV),
            (dict(_5=40), UNS), (dict(_5=272), UNS), (dict(_8=None), INV), (dict(_0=None), INV), (dict(_14=None), INV),
            (dict(_16=None), INV), (dict(_6=None), INV), (dict(_0=ODD4), MIS), (dict(_6=ODD), MIS), (dict(_8=ODD), MIS),
            (dict(_14=ODD), MIS), (dict(_15=ODD), MIS), (dict(_16=ODD), MIS), (dict(_10=ODD), MIS), (dict(_12=ODD), MIS),
            (dict(_2=1 << 16, _7=1 << 16), UNS)]:
        assert call(*changed(ok, **change)) == status, change
    assert call(*changed(ok, _2=0)) == OK and call(*changed(ok, _7=0)) == OK
    #       w    B  N   ne    bud rec idx   kept  stream
    ok = [FAKE, 2, 50, None, 10, 2, FAKE, None, None]
    call = lib.csa_evict
    for change, status in [(dict(_0=None), INV), (dict(_1=-1), INV), (dict(_2=-1), INV), (dict(_4=-1), INV), (dict(_5=-1), INV),
                           (dict(_6=None), INV), (dict(_0=ODD), MIS), (dict(_3=ODD), MIS), (dict(_6=ODD), MIS), (dict(_7=ODD), MIS),
                           (dict(_2=(1 << 30) + 1), UNS)]:
        assert call(*changed(ok, **change)) == status, change
    assert call(*changed(ok, _1=0)) == OK


def test_injected_launch_failures_surface(lib):
    f = (ctypes.c_double * 16)()
    calls = [
        lambda: lib.csa_rope(FAKE, FAKE, 2, None, None, None, 0, None, 1, 1, 4, 64, 32, 0, 1, f, 1.0, None, 0, 1, 0, None),
        lambda: lib.hca_dense_attn_prefix(FAKE, 1, 2, 1, 64, 128, FAKE, 100, FAKE, 10, None, 4, FAKE, 16, None, None, 16,
                                          None, 0.0, FAKE, None, FAKE, 1 << 40, None),
        lambda: lib.hca_entry_weights(FAKE, 1, 2, 1, 64, 128, FAKE, 50, None, 0, None, 4, None, 0.0, FAKE, None, FAKE, None),
        lambda: lib.csa_evict(FAKE, 2, 50, None, 10, 2, FAKE, None, None)]
    for call in calls:
        assert lib.csa_debug_inject_launch_error(719) == OK
        assert call() == api.CSA_ERR_CUDA
    assert lib.csa_evict(FAKE, 0, 50, None, 10, 2, FAKE, None, None) == OK


def test_dependent_kernels_wait_before_they_read_an_array():
    # a kernel launched while the one before it ends sees that one's writes only behind its wait:
    # what stands above it in the source sets up shared memory, barriers and TMEM
    reads = re.compile(r"\ba\.\w+ ?\[|\ba\.\w+ \+|__ldg|row_keys\(|cp_async16\(|tma_load|load_q\(|\berr\)|issue_tma\((?!int)"
                       r"|fill_\w+[<(]|entries_of\(")
    waiting = 0
    for path in sorted(glob.glob(os.path.join(build_mod.CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path, encoding="utf-8").read())
        for kernel in re.split(r"__global__", text)[1:]:
            body = kernel[kernel.index("{"):]
            end = re.search(r"\n}", body)
            body = body[:end.start()] if end else body
            at = re.search(r"grid_wait\(\)|griddepcontrol\.wait", body)
            if at is None:
                continue
            waiting += 1
            head = re.sub(r"auto \w+ = \[&\].*?\n    };", "", body[:at.start()], flags=re.S)    # (defined, called later)
            early = reads.search(head)
            assert early is None, (os.path.basename(path), early.group(0))
    assert waiting >= 12


def test_binding_checks_shapes():
    z = torch.zeros
    with pytest.raises(ValueError, match="one dtype"):
        api.hca_attn_prefix(z(1, 1, 64, 128), z(4, 128).bfloat16(), z(1, 2, 128), 4, z(1, 2, 128), 2)
    with pytest.raises(ValueError, match="one dtype"):
        api.entry_weights(z(1, 1, 64, 128), z(1, 4, 128).bfloat16(), 4, z(1, 1, 64))
    with pytest.raises(ValueError, match="CUDA"):
        api.evict(z(2, 4), 2)
    with pytest.raises(ValueError, match="B, N_cap"):
        api.csa_evict(z(4), 2, z(1, 2))


# ------------------------------------------------------------------ the definitions themselves
def test_reference_attention_against_torch():
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(3, 16, generator=g, dtype=torch.float64), torch.randn(9, 16, generator=g, dtype=torch.float64)
    out, lse, bound, _ = ref.attention_row(q, k, 0.25, torch.float32)
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], k[None], scale=0.25)[0]
    assert float((out - want).abs().max()) < 1e-12 and float(bound.max()) < 1e-4
    a = dict(q=q.reshape(1, 1, 3, 16), kv_p=k[:4], kv_c=k[None, 4:7], m=2, kv_raw=k[None, 7:], window=2, n_entries=None,
             raw_pos0=torch.tensor([12]), raw_len=None, q_pos=torch.tensor([[13]]), scale=0.25)
    assert float((ref.prefix_attention(a, torch.float32)[0][0, 0] - want).abs().max()) < 1e-12
    a["q_pos"] = torch.tensor([[9]])        # 5 entries, and no raw row at a position <= 9
    got = ref.prefix_attention(a, torch.float32)[0][0, 0]
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None, :5], k[None, :5], scale=0.25)[0]
    assert float((got - want).abs().max()) < 1e-12


def test_reference_evict_by_hand():
    w = torch.tensor([[3.0, 1.0, 3.0, -1.0, 2.0, 0.5, 9.0]])
    idx, kept, out = ref.evict(w, [6], 3, 1)       # entry 5 is recent; then 0 and 2 (equal, lower index first)
    assert idx.tolist() == [[0, 2, 5]] and kept.tolist() == [3]
    assert out.tolist() == [[3.0, -1.0, 3.0, -1.0, -1.0, 0.5, 9.0]]


def test_reference_weights_by_hand():
    q, kv = torch.ones(1, 1, 2, 4), torch.stack([torch.zeros(4), torch.ones(4)])[None]
    w, bound = ref.entry_weights(q, kv, 1, torch.zeros(1, 1, 2), torch.tensor([[1.0, 0.0]]), None, None, torch.tensor([[1]]))
    assert abs(float(w[0, 0]) - 3.0) < 1e-12 and abs(float(w[0, 1]) - 2 * math.e ** 2) < 1e-12
    assert float(bound.max()) < 1e-4
