"""Refusals of the microscaled 4-bit and expert entry points, on the CPU: bad
arguments are reported before any HIP call, by the C functions and by the
binding's own checks."""

import ctypes

import pytest

import weight_only_lut_amd as lutq
from weight_only_lut_amd import _mx

torch = pytest.importorskip("torch")

OK, EINVAL, EGROUP, EALIGN, EMISMATCH, ESIZE, EUNSUP = 0, -1, -3, -4, -5, -6, -8
P = 1 << 20      # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    return lutq.load_library()


def test_quantize_refuses(lib):
    def q(x=P, dtype=0, rows=2, K=64, ldx=64, rule=0, codes=P, scales=P):
        return lib.lutq_mx_quantize(x, dtype, rows, K, ldx, rule, codes, scales, None)
    assert q(rows=0) == OK and q(K=0, ldx=0) == OK
    assert q(x=None) == q(codes=None) == q(scales=None) == EINVAL
    assert q(dtype=3) == q(rule=2) == q(rows=-1) == q(K=-32) == q(ldx=32) == EINVAL
    assert q(K=48) == EGROUP
    assert q(x=P + 8) == q(codes=P + 2) == q(dtype=1, ldx=68) == q(ldx=65) == EALIGN
    assert q(K=(1 << 20) + 32, ldx=1 << 21) == EUNSUP
    assert q(rows=(1 << 31) - 1, K=1 << 20, ldx=1 << 20) == EUNSUP


def test_dequantize_refuses(lib):
    def d(codes=P, scales=P, dtype=0, rows=2, K=64, x=P):
        return lib.lutq_mx_dequantize(codes, scales, dtype, rows, K, x, None)
    assert d(rows=0) == OK
    assert d(x=None) == d(codes=None) == d(scales=None) == d(dtype=5) == d(rows=-1) == EINVAL
    assert d(K=40) == EGROUP
    assert d(codes=P + 1) == d(x=P + 8) == EALIGN


def _desc(E=1, N=48, K=64, **over):
    d = _mx.MxPackedDesc(0x34584D4C, 1, E, N, K, 0, lutq.load_library().lutq_mx_packed_bytes(E, N, K), P)
    for k, v in over.items():
        setattr(d, k, v)
    return d


def test_pack_refuses(lib):
    out = _mx.MxPackedDesc()
    need = lib.lutq_mx_packed_bytes(2, 48, 64)
    # 2 experts x 3 tiles x (one 1 KiB block, one quad of scales, 16 fp32)
    assert need == 2 * 3 * (1024 + 256 + 64)

    def p(codes=P, scales=2 * P, E=2, N=48, K=64, dst=3 * P, n=need, o=ctypes.addressof(out)):
        return lib.lutq_mx_pack(codes, scales, E, N, K, dst, n, o, None)
    assert p(o=None) == p(codes=None) == p(scales=None) == p(dst=None) == p(E=0) == p(N=-1) == EINVAL
    assert p(K=33) == EGROUP
    assert p(codes=P + 8) == p(dst=3 * P + 4) == EALIGN
    assert p(n=need - 1) == ESIZE
    assert p(E=1025) == p(N=(1 << 24) + 1) == p(K=(1 << 20) + 32) == EUNSUP
    assert p(dst=P + 1024) == p(dst=2 * P) == EINVAL       # overlaps its inputs
    assert p(N=0) == OK and out.nbytes == 0
    assert lib.lutq_mx_packed_bytes(1, 16, 33) == lib.lutq_mx_packed_bytes(0, 16, 32) == 0


def test_matmul_refuses(lib):
    def m(x=P, dtype=2, ldx=64, desc=None, y=P, M=2, N=48, K=64, path=0, **over):
        d = desc or _desc(**over)
        return lib.lutq_mx_matmul(x, dtype, ldx, ctypes.addressof(d), y, M, N, K, path, None, 0, None)
    assert m(M=0) == OK
    assert m(x=None) == m(y=None) == m(dtype=0) == m(path=3) == m(M=-1) == m(ldx=63) == EINVAL
    assert m(N=47) == m(K=32) == m(magic=0) == m(version=2) == m(nbytes=16) == EMISMATCH
    assert m(desc=_desc(E=2)) == EMISMATCH
    assert m(data=None) == EINVAL
    assert m(x=P + 2) == m(y=P + 4) == m(ldx=66) == m(data=P + 8) == EALIGN
    assert lib.lutq_mx_matmul(P, 2, 64, None, P, 1, 48, 64, 0, None, 0, None) == EINVAL
    assert m(ldx=(1 << 22) + 8) == EUNSUP

    # a tall split of a small matrix keeps its results in the caller's workspace
    split = lib.lutq_mx_workspace_bytes(96, 48, 4096, 0, 0)
    assert split > 0 and lib.lutq_mx_workspace_bytes(96, 48, 4096, 0, 1) == 0
    d = _desc(K=4096)
    def ms(ws, n):
        return lib.lutq_mx_matmul(P, 2, 4096, ctypes.addressof(d), P, 96, 48, 4096, 0, ws, n, None)
    assert ms(None, 0) == EINVAL and ms(P, split - 1) == ESIZE and ms(P + 8, split) == EALIGN

    # few 4-bit rows are decoded beside the weights, more need their scales in tile order
    need = lib.lutq_mx_workspace_bytes(40, 48, 64, 1, 0)
    assert lib.lutq_mx_workspace_bytes(2, 48, 64, 1, 0) == 0 == lib.lutq_mx_workspace_bytes(40, 48, 63, 1, 0)
    assert need > 0 and lib.lutq_mx_workspace_bytes(0, 48, 64, 1, 0) == 0

    def m4(xc=P, xs=P, y=P, dtype=2, M=40, N=48, K=64, ws=P, n=need, **over):
        d = _desc(**over)
        return lib.lutq_mx_matmul_mx(xc, xs, ctypes.addressof(d), y, dtype, M, N, K, ws, n, None)
    assert m4(M=0) == OK
    assert m4(xc=None) == m4(xs=None) == m4(y=None) == m4(dtype=0) == m4(M=-2) == EINVAL
    assert m4(N=16) == m4(K=96) == EMISMATCH
    assert m4(xc=P + 8) == m4(y=P + 2) == m4(ws=P + 8) == EALIGN
    assert m4(ws=None) == EINVAL and m4(n=need - 1) == ESIZE


def _opts(**over):
    o = _mx.MoeOptions(0, 1, 1, 1, 1, 1.0)
    for k, v in over.items():
        setattr(o, k, v)
    return o


def test_route_refuses(lib):
    def r(logits=P, dtype=0, ld=16, bias=None, T=2, E=16, k=4, ids=P, w=P, plan=P, **over):
        o = _opts(**over)
        return lib.lutq_moe_route(logits, dtype, ld, bias, T, E, k, ctypes.addressof(o), ids, w, plan, None)
    assert r(T=0, plan=None) == OK
    assert r(logits=None) == r(ids=None) == r(w=None) == r(dtype=3) == r(ld=15) == EINVAL
    assert r(k=0) == r(k=17) == r(E=0) == r(T=-1) == EINVAL
    assert r(E=1025, ld=1025) == r(E=64, ld=64, k=33) == r(T=1 << 23, k=4) == EUNSUP
    assert r(score=2) == r(groups=0) == r(groups=3) == r(top_groups=0) == r(top_groups=2) == EINVAL
    assert r(group_best=0) == r(group_best=3) == r(groups=16, group_best=2) == r(renorm=2) == EINVAL
    assert r(scale=float("nan")) == EINVAL
    assert r(E=128, ld=128, groups=128) == EUNSUP
    assert r(logits=P + 2) == r(dtype=1, logits=P + 1) == r(bias=P + 2) == r(ids=P + 2) == r(w=P + 1) == EALIGN
    assert r(plan=P + 2) == EALIGN
    assert lib.lutq_moe_plan_ints(4, 16, 17) == 0 and lib.lutq_moe_plan_ints(-1, 16, 2) == 0
    assert lib.lutq_moe_plan_ints(4, 16, 2) >= 16 + 1 + 8
    assert lib.lutq_moe_plan(None, 2, 16, 4, P, None) == lib.lutq_moe_plan(P, 2, 16, 4, None, None) == EINVAL
    assert lib.lutq_moe_plan(P + 1, 2, 16, 4, P, None) == EALIGN


def test_moe_mlp_refuses(lib):
    E, D, F = 4, 96, 64
    need = lib.lutq_moe_workspace_bytes(2, 2, D, F)
    assert need > 0 and lib.lutq_moe_workspace_bytes(2, 33, D, F) == 0

    def m(x=P, dtype=2, ldx=D, gu=None, dn=None, ids=P, w=P, plan=P, T=2, k=2, ws=P, n=need, y=P):
        gu, dn = gu or _desc(E, 2 * F, D), dn or _desc(E, D, F)
        return lib.lutq_moe_mlp(x, dtype, ldx, ctypes.addressof(gu), ctypes.addressof(dn), ids, w, plan, T, k,
                                ws, n, y, None)
    assert m(T=0) == OK
    assert m(x=None) == m(ids=None) == m(w=None) == m(plan=None) == m(ws=None) == m(y=None) == EINVAL
    assert m(dtype=0) == m(ldx=D - 8) == m(k=0) == m(k=5) == m(T=-1) == EINVAL
    assert m(dn=_desc(E, D, 32)) == m(dn=_desc(E + 1, D, F)) == m(gu=_desc(E, F, D)) == EMISMATCH
    assert m(gu=_desc(E, 2 * F, D, magic=1)) == EMISMATCH
    assert m(x=P + 8) == m(ldx=D + 4) == m(y=P + 2) == m(ws=P + 8) == m(ids=P + 2) == EALIGN
    assert m(n=need - 1) == ESIZE


def test_binding_checks_before_calling():
    """Types, shapes and strides are refused before the library is called (here
    on CPU tensors, which are then refused for not being on the GPU)."""
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x = torch.zeros((2, 64), dtype=bf16)
    w = lutq.MxPacked(torch.zeros(8192, dtype=u8), _desc())
    gu = lutq.MxPacked(torch.zeros(8192, dtype=u8), _desc(4, 128, 96))
    dn = lutq.MxPacked(torch.zeros(8192, dtype=u8), _desc(4, 96, 64))
    codes, scales = torch.zeros((2, 32), dtype=u8), torch.zeros((2, 2), dtype=u8)
    r = lutq.Routing(torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 2)), torch.zeros(64, dtype=torch.int32), 4)
    xd = torch.zeros((2, 96), dtype=bf16)
    values = [
        lambda: lutq.mx_quantize(torch.zeros(2, 48)), lambda: lutq.mx_quantize(x, rule="up"),
        lambda: lutq.mx_quantize(x.view(2, 2, 32)), lambda: lutq.mx_quantize(torch.zeros(64, 64).t()[:, ::2]),
        lambda: lutq.mx_dequantize(codes, scales[:, :1].contiguous()),
        lambda: lutq.mx_pack(codes.view(1, 1, 2, 32), scales.view(1, 1, 2, 2)),
        lambda: lutq.mx_matmul(torch.zeros((2, 32), dtype=bf16), w), lambda: lutq.mx_matmul(x, w, path="fast"),
        lambda: lutq.mx_matmul(x, gu), lambda: lutq.mx_matmul((codes, scales), w, path="tile"),
        lambda: lutq.mx_matmul(x, w, out=torch.zeros((2, 47), dtype=bf16)),
        lambda: lutq.moe_route(x, 2, score="max"), lambda: lutq.moe_route(x, 2, bias=torch.zeros(63)),
        lambda: lutq.moe_mlp(x, gu, dn, r), lambda: lutq.moe_mlp(xd, dn, gu, r),
        lambda: lutq.moe_mlp(xd[:1], gu, dn, r),
        lambda: lutq.moe_plan(r.ids.view(-1), r.weights.view(-1), 4),
    ]
    for f in values:
        with pytest.raises(ValueError):
            f()
    types = [
        lambda: lutq.mx_quantize(x.int()), lambda: lutq.mx_matmul(x.float(), w), lambda: lutq.mx_matmul(x, x),
        lambda: lutq.mx_matmul(x, w, dtype=f32), lambda: lutq.mx_matmul((codes, scales), w, dtype=f32),
        lambda: lutq.mx_dequantize(codes.int(), scales), lambda: lutq.mx_dequantize(codes, scales, torch.int32),
        lambda: lutq.moe_route(x.int(), 2), lambda: lutq.moe_route(x, 2, bias=torch.zeros(64, dtype=bf16)),
        lambda: lutq.moe_mlp(xd, gu, dn, None), lambda: lutq.moe_mlp(xd.float(), gu, dn, r),
        lambda: lutq.moe_plan(r.ids.long(), r.weights, 4),
        # all as they should be, but not on a GPU
        lambda: lutq.mx_quantize(x), lambda: lutq.mx_matmul(x, w), lambda: lutq.moe_route(x, 2),
        lambda: lutq.mx_dequantize(codes, scales), lambda: lutq.mx_pack(codes, scales),
        lambda: lutq.mx_matmul((codes, scales), w), lambda: lutq.moe_mlp(xd, gu, dn, r),
        lambda: lutq.moe_plan(r.ids, r.weights, 4),
    ]
    for f in types:
        with pytest.raises(TypeError):
            f()
