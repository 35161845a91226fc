"""CPU tests of the expert-layer operators: every refusal is made before anything
reaches the GPU, by the C entry points (with pointers that must not be followed)
and by the Python checks; and the oracle's pins."""
import ctypes

import numpy as np
import pytest
import torch

import newton_schulz_gram_amd as nsg
from oracle import expert_oracle as ref

P16 = 0x10000  # an aligned address that no call may follow
OK, ARG, DTYPE, SHAPE, WORKSPACE = 0, 1, 2, 3, 4


def sort(ids=P16, bits=64, T=4, k=2, E=8, offsets=P16, rows=P16, tokens=P16, ws=None, n=0):
    return nsg.lib().nsg_expert_sort(ids, bits, T, k, E, offsets, rows, tokens, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bits=16), DTYPE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE),
    (dict(T=1 << 25, k=2), SHAPE), (dict(k=1 << 40), SHAPE), (dict(ids=None), ARG), (dict(offsets=None), ARG),
    (dict(rows=None), ARG), (dict(tokens=None), ARG), (dict(ids=P16 + 4), ARG), (dict(rows=P16 + 2), ARG),
    (dict(T=70000), WORKSPACE), (dict(T=70000, ws=P16, n=64), WORKSPACE), (dict(T=70000, ws=P16 + 1, n=1 << 30), WORKSPACE),
])
def test_sort_refusals(kw, code):
    assert sort(**kw) == code


def test_sort_workspace_size():
    assert nsg.expert_sort_workspace_size(1, 8, 512) == 0
    assert nsg.expert_sort_workspace_size(0, 8, 512) == 0
    big = nsg.expert_sort_workspace_size(16384, 8, 512)
    assert big > 0 and big % (4 * 512) == 0
    assert nsg.lib().nsg_expert_sort_workspace_size(1, 1, 1, None) == ARG


def dispatch(x=P16, dt=1, T=4, C=8, ld=8, offsets=P16, E=3, rows=P16, k=2, out=P16):
    return nsg.lib().nsg_expert_dispatch(x, dt, T, C, ld, offsets, E, rows, k, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), DTYPE), (dict(dt=-1), DTYPE), (dict(T=-1), SHAPE), (dict(C=70000, ld=70000), SHAPE), (dict(ld=7), SHAPE),
    (dict(k=0), SHAPE), (dict(T=1 << 25, k=2), SHAPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(x=None), ARG),
    (dict(offsets=None), ARG), (dict(rows=None), ARG), (dict(out=None), ARG), (dict(x=P16 + 1), ARG), (dict(out=P16 + 1), ARG),
    (dict(rows=P16 + 2), ARG), (dict(T=0), OK), (dict(C=0, ld=0), OK),
])
def test_dispatch_refusals(kw, code):
    assert dispatch(**kw) == code


def combine(y=P16, dt=1, P=8, C=8, ld=8, rows=P16, T=4, k=2, w=P16, out=P16):
    return nsg.lib().nsg_expert_combine(y, dt, P, C, ld, rows, T, k, w, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=4), DTYPE), (dict(k=0), SHAPE), (dict(T=-2), SHAPE), (dict(P=-1), SHAPE), (dict(ld=4), SHAPE), (dict(y=None), ARG),
    (dict(rows=None), ARG), (dict(out=None), ARG), (dict(w=P16 + 2), ARG), (dict(y=P16 + 1), ARG), (dict(T=0), OK),
])
def test_combine_refusals(kw, code):
    assert combine(**kw) == code


def backward(dout=P16, lddo=8, y=P16, ldy=8, dt=1, P=8, C=8, offsets=P16, E=3, rows=P16, T=4, k=2, w=None, dy=P16, dw=P16):
    return nsg.lib().nsg_expert_combine_backward(dout, lddo, y, ldy, dt, P, C, offsets, E, rows, T, k, w, dy, dw, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), DTYPE), (dict(P=7), SHAPE), (dict(E=0), SHAPE), (dict(E=2000), SHAPE), (dict(lddo=4), SHAPE), (dict(ldy=4), SHAPE),
    (dict(dout=None), ARG), (dict(y=None), ARG), (dict(offsets=None), ARG), (dict(rows=None), ARG), (dict(dy=None), ARG),
    (dict(dw=None), ARG), (dict(dw=P16 + 1), ARG), (dict(dy=P16 + 1), ARG), (dict(T=0, P=0), OK),
])
def test_backward_refusals(kw, code):
    assert backward(**kw) == code


def quantize(x=P16, dt=1, B=1, R=4, C=8, ld=8, block=0, f8=3, q=P16, s=P16, qt=None, st=None):
    return nsg.lib().nsg_quantize_fp8(x, dt, B, R, C, ld, block, f8, q, s, qt, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), DTYPE), (dict(f8=1), DTYPE), (dict(f8=5), DTYPE), (dict(block=2), ARG), (dict(B=-1), SHAPE), (dict(B=70000), SHAPE),
    (dict(R=-1), SHAPE), (dict(ld=7), SHAPE), (dict(R=(1 << 25) + 1), SHAPE), (dict(block=1, R=128 * 65535 + 1), SHAPE),
    (dict(qt=P16, st=P16), ARG), (dict(block=1, qt=P16), ARG), (dict(block=1, st=P16), ARG), (dict(x=None), ARG), (dict(q=None), ARG),
    (dict(s=None), ARG), (dict(q=P16 + 8), ARG), (dict(block=1, qt=P16 + 8, st=P16), ARG), (dict(x=P16 + 1), ARG), (dict(B=0), OK),
    (dict(R=0), OK), (dict(C=0, ld=0), OK),
])
def test_quantize_refusals(kw, code):
    assert quantize(**kw) == code


def columns(x=P16, dt=1, R=8, C=8, ld=8, offsets=P16, E=2, tokens=None, P=8, f8=4, q=P16, s=P16):
    return nsg.lib().nsg_quantize_fp8_columns(x, dt, R, C, ld, offsets, E, tokens, P, f8, q, s, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=4), DTYPE), (dict(f8=0), DTYPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(P=7), SHAPE), (dict(P=-1, tokens=P16), SHAPE),
    (dict(ld=7), SHAPE), (dict(x=None), ARG), (dict(offsets=None), ARG), (dict(q=None), ARG), (dict(s=None), ARG), (dict(q=P16 + 4), ARG),
    (dict(tokens=P16 + 1, P=9), ARG), (dict(C=0, ld=0), OK),
])
def test_columns_refusals(kw, code):
    assert columns(**kw) == code


def gemm(ad=3, bd=3, od=1, batch=1, M=4, N=8, K=128, qa=P16, sa=P16, ab=0, qb=P16, sb=P16, bb=1, out=P16):
    return nsg.lib().nsg_gemm_fp8_nt(ad, bd, od, batch, M, N, K, qa, sa, ab, qb, sb, bb, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ad=1), DTYPE), (dict(bd=0), DTYPE), (dict(od=3), DTYPE), (dict(K=100), SHAPE), (dict(K=0), SHAPE), (dict(K=-128), SHAPE),
    (dict(M=-1), SHAPE), (dict(N=70000), SHAPE), (dict(batch=-1), SHAPE), (dict(batch=65536), SHAPE), (dict(ab=2), ARG), (dict(bb=-1), ARG),
    (dict(qa=None), ARG), (dict(sa=None), ARG), (dict(qb=None), ARG), (dict(sb=None), ARG), (dict(out=None), ARG), (dict(qa=P16 + 8), ARG),
    (dict(qb=P16 + 8), ARG), (dict(sa=P16 + 2), ARG), (dict(out=P16 + 1), ARG), (dict(M=0), OK), (dict(N=0), OK), (dict(batch=0), OK),
    (dict(M=1 << 25, N=65536, batch=64), SHAPE),
])
def test_gemm_refusals(kw, code):
    assert gemm(**kw) == code


def expert_gemm(ad=3, bd=3, od=1, T=4, P=8, E=2, N=8, K=128, qa=P16, sa=P16, tokens=P16, qb=P16, sb=P16, bb=1, offsets=P16, out=P16):
    return nsg.lib().nsg_expert_gemm_fp8(ad, bd, od, T, P, E, N, K, qa, sa, tokens, qb, sb, bb, offsets, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ad=2), DTYPE), (dict(od=4), DTYPE), (dict(E=0), SHAPE), (dict(E=1025), SHAPE), (dict(T=0), SHAPE), (dict(tokens=None), SHAPE),
    (dict(K=64), SHAPE), (dict(P=-1), SHAPE), (dict(bb=3), ARG), (dict(offsets=None), ARG), (dict(qa=None), ARG), (dict(out=None), ARG),
    (dict(tokens=P16 + 2), ARG), (dict(P=0), OK), (dict(N=0), OK),
])
def test_expert_gemm_refusals(kw, code):
    assert expert_gemm(**kw) == code


def wgrad(ad=4, bd=3, od=2, P=200, E=2, N=8, K=16, qa=P16, sa=P16, qb=P16, sb=P16, offsets=P16, out=P16):
    return nsg.lib().nsg_expert_wgrad_fp8(ad, bd, od, P, E, N, K, qa, sa, qb, sb, offsets, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(ad=1), DTYPE), (dict(bd=7), DTYPE), (dict(od=3), DTYPE), (dict(P=-1), SHAPE), (dict(E=0), SHAPE), (dict(N=70000), SHAPE),
    (dict(K=70000), SHAPE), (dict(qa=None), ARG), (dict(offsets=None), ARG), (dict(qb=P16 + 4), ARG), (dict(out=P16 + 2), ARG),
    (dict(N=0), OK), (dict(K=0), OK),
])
def test_wgrad_refusals(kw, code):
    assert wgrad(**kw) == code


def test_fp8_columns():
    assert nsg.fp8_columns(0, 1) == 128 and nsg.fp8_columns(127, 3) == 384 and nsg.fp8_columns(128, 3) == 512
    cap = ctypes.c_int64(0)
    assert nsg.lib().nsg_fp8_columns(-1, 1, ctypes.byref(cap)) == SHAPE
    assert nsg.lib().nsg_fp8_columns(1, 1025, ctypes.byref(cap)) == SHAPE
    assert nsg.lib().nsg_fp8_columns(1, 1, None) == ARG


def test_fp8_columns_hold_every_split():
    """floor(P / 128) + E blocks suffice for any lengths that add up to P."""
    g = np.random.default_rng(0)
    for _ in range(2000):
        P, E = int(g.integers(0, 2000)), int(g.integers(1, 40))
        o = np.concatenate([[0], np.sort(g.integers(0, P + 1, size=E - 1)), [P]])
        assert sum(-(-int(n) // 128) for n in np.diff(o)) * 128 <= nsg.fp8_columns(P, E)


def test_existing_calls_refuse_8_bit_types():
    L = nsg.lib()
    for d in (3, 4):
        assert L.ns_muon_momentum(P16, 2, P16, d, 8, 0.5, None) == DTYPE
        assert L.nsg_gemm_nt(d, 0, 1, 256, 256, 256, P16, 256, 0, P16, 256, 0, 1.0, 0.0, None, 0, P16, 256, None, 0, None, 0.0, 0,
                             None, None) == DTYPE


def test_python_refuses_cpu_tensors():
    x = torch.zeros(4, 8)
    i = torch.zeros((4, 2), dtype=torch.int64)
    plan = nsg.ExpertPlan(*(torch.zeros(n, dtype=torch.int32) for n in (3, (4, 2), 8)))
    q, s = torch.zeros((4, 128)).to(torch.float8_e4m3fn), torch.zeros((1, 4))
    for call in (lambda: nsg.expert_sort(i, 4), lambda: nsg.expert_dispatch(x, plan), lambda: nsg.expert_combine(x, plan),
                 lambda: nsg.expert_combine_backward(x, x, plan), lambda: nsg.quantize_fp8(x),
                 lambda: nsg.quantize_fp8_columns(x, plan.offsets), lambda: nsg.gemm_fp8_nt(q, s, q, s),
                 lambda: nsg.expert_gemm_fp8(q, s, q[None], s[None], plan.offsets),
                 lambda: nsg.expert_wgrad_fp8(q, s, q, s, plan.offsets)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.parametrize("f8,dt", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_oracle_rounding_is_the_type_s(f8, dt):
    """The oracle's rounding gives every number of the type back, and torch's cast
    everywhere in between (ties included)."""
    grid = torch.arange(256, dtype=torch.uint8).view(dt).float().double().numpy()
    grid = np.unique(grid[np.isfinite(grid)])
    assert np.array_equal(ref.round8(grid, f8), grid)
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([mid, np.random.default_rng(1).uniform(grid[0], grid[-1], 5000), np.random.default_rng(2).standard_normal(5000)])
    v = v.astype(np.float32)
    assert np.array_equal(ref.round8(v, f8), torch.from_numpy(v).to(dt).float().double().numpy())
    assert np.isnan(ref.round8(np.array([np.inf, np.nan]), "e4m3")).all() and np.isinf(ref.round8(np.array([-np.inf]), "e5m2")).all()


def test_oracle_sort_pins():
    o, r, t = ref.expert_sort(np.array([[2, 0], [0, -1], [2, 5]]), 3)
    assert o.tolist() == [0, 2, 2, 4] and r.tolist() == [[2, 0], [1, -1], [3, -1]] and t.tolist() == [0, 1, 0, 2, -1, -1]
