"""Host-only checks of the 4-bit operators (no GPU needed): arguments that the C ABI and the
binding refuse before any launch, the valid no-ops, and the workspace's size."""
import ctypes

import pytest
import torch

import bit_moe_routed_b200 as bm
from bit_moe_routed_b200 import build as bm_build

P = ctypes.c_void_p
A = 1 << 20  # an aligned address that is never read: every call here is refused first


@pytest.fixture(scope="module")
def L():
    bm_build.build()
    return bm.lib()


def mat(codes=A, scales=A, zeros=None):
    return bm._W4Matrix(codes, scales, zeros)


def gemm(L, x=A, dtype=0, M=4, w=None, N=64, K=256, group=128, C=A):
    w = mat() if w is None else w
    return L.moe_w4_gemm(P(x), dtype, M, ctypes.byref(w), N, K, group, P(C), None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(M=65), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0), dict(K=192),
    dict(K=-128), dict(K=(1 << 20) + 128), dict(group=16), dict(group=0), dict(group=256),
    dict(dtype=2), dict(dtype=-1), dict(x=0), dict(x=A + 8), dict(C=0), dict(C=A + 2),
    dict(w=mat(codes=None)), dict(w=mat(codes=A + 8)), dict(w=mat(scales=None)),
    dict(w=mat(scales=A + 1))], ids=str)
def test_gemm_refuses(L, bad):
    assert gemm(L, **bad) == bm.MOE_ERR_INVALID_ARG
    assert L.moe_last_error()


def test_gemm_without_weights_or_rows(L):
    assert L.moe_w4_gemm(P(A), 0, 1, None, 64, 256, 128, P(A), None) == bm.MOE_ERR_INVALID_ARG
    assert gemm(L, M=0, x=0, C=0) == bm.MOE_OK  # no rows: a no-op
    assert gemm(L, M=0, K=192) == bm.MOE_ERR_INVALID_ARG  # of valid sizes


def layer(L, T=4, k=2, scores=A, x=A, idx=A, tw=A, out=A, ws=A, ws_bytes=1 << 30, zeros=None,
          down_zeros="same", **w):
    f = dict(E=8, d=256, f=128, group=32, dtype=0, shared=1)
    f.update(w)
    dz = zeros if down_zeros == "same" else down_zeros
    st = bm._W4Weights(mat(zeros=zeros), mat(zeros=zeros), mat(zeros=dz), *f.values())
    return L.moe_forward_w4(P(scores), P(x), T, k, ctypes.byref(st), P(idx), P(tw), P(out), P(ws),
                            ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(T=65), dict(k=0), dict(k=9), dict(k=33, E=64), dict(E=0), dict(E=1025),
    dict(d=0), dict(d=80), dict(d=96, group=64), dict(d=16384 + 32), dict(f=48),
    dict(f=96, group=64), dict(f=16384 + 32), dict(group=48), dict(dtype=2), dict(shared=2),
    dict(shared=-1), dict(down_zeros=A), dict(scores=0), dict(x=0), dict(x=A + 8), dict(idx=0),
    dict(tw=0), dict(out=0), dict(out=A + 4), dict(ws=0), dict(ws=A + 128)], ids=str)
def test_layer_refuses(L, bad):
    assert layer(L, **bad) == bm.MOE_ERR_INVALID_ARG
    assert L.moe_last_error()


def test_layer_workspace(L):
    size = L.moe_w4_workspace_size
    need = size(4, 2, 8, 256, 128, 1)
    assert need >= 12 * (128 * 4 + 256 * 4)  # h's two terms and y of 12 rows
    assert layer(L, ws_bytes=need - 1) == bm.MOE_ERR_WORKSPACE
    assert b"needs" in L.moe_last_error()
    assert size(4, 2, 8, 256, 128, 0) < need
    for sizes in [(65, 2, 8, 256, 128, 1), (4, 9, 8, 256, 128, 1), (4, 2, 0, 256, 128, 1),
                  (4, 2, 8, 80, 128, 1), (4, 2, 8, 256, 100, 1), (4, 2, 8, 256, 128, 2),
                  (-1, 2, 8, 256, 128, 1)]:
        assert size(*sizes) == 0
    assert layer(L, T=0, scores=0, x=0, idx=0, tw=0, out=0, ws=0, ws_bytes=0) == bm.MOE_OK


def tensors(lead=(), N=64, K=256, G=32, dtype=torch.bfloat16, zeros=True):
    return (torch.zeros((*lead, N, K // 2), dtype=torch.uint8),
            torch.ones((*lead, N, K // G), dtype=dtype),
            torch.full((*lead, N, K // G), 8, dtype=torch.uint8) if zeros else None)


def test_matrix_descriptor():
    m = bm.W4Matrix(*tensors())
    assert (m.N, m.K, m.group, m.dtype) == (64, 256, 32, torch.bfloat16)
    assert m.struct().codes == m.codes.data_ptr() and m.struct().zeros == m.zeros.data_ptr()
    assert bm.W4Matrix(*tensors(zeros=False)).struct().zeros is None
    c, s, z = tensors()
    for args in [(c.int(), s, z), (c, s.float(), z), (c, s[:-1], z), (c, s[:, :-1], z),
                 (c, s, z.int()), (c, s, z[:-1]), (c[0], s[0], None),
                 (c, torch.ones((64, 1), dtype=torch.bfloat16), None),
                 (c, torch.ones((64, 16), dtype=torch.bfloat16), None)]:
        with pytest.raises(ValueError):
            bm.W4Matrix(*args)
    with pytest.raises(ValueError):  # strides are not taken
        bm.W4Matrix(c.t().contiguous().t(), s, z).struct()


def test_layer_descriptor():
    up = dict(lead=(5,), N=64, K=256)
    down = dict(lead=(5,), N=256, K=64)
    g = bm.W4Matrix(*tensors(**up))
    w = bm.W4Layer(g, bm.W4Matrix(*tensors(**up)), bm.W4Matrix(*tensors(**down)))
    assert (w.E, w.d, w.f, w.group) == (4, 256, 64, 32) and w.struct().shared == 1
    w0 = bm.W4Layer(g, g, bm.W4Matrix(*tensors(**down)), shared=False)
    assert w0.E == 5 and w0.struct().shared == 0
    for d in [dict(zeros=False), dict(G=64), dict(dtype=torch.float16), dict(lead=(4,)),
              dict(N=128), dict(K=128), dict(lead=())]:
        with pytest.raises(ValueError):
            bm.W4Layer(g, g, bm.W4Matrix(*tensors(**{**down, **d})))
    one = dict(lead=(1,))
    with pytest.raises(ValueError):  # only a shared expert
        bm.W4Layer(bm.W4Matrix(*tensors(**{**up, **one})), bm.W4Matrix(*tensors(**{**up, **one})),
                   bm.W4Matrix(*tensors(**{**down, **one})))


def test_calls_refuse_tensors_that_do_not_fit():
    """Shapes, types and devices: tensors on the host are refused, not read."""
    m = bm.W4Matrix(*tensors())
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    for bad in [x.half(), x[:, :128], x[0], x]:
        with pytest.raises(ValueError):
            bm.w4_gemm(bad, m)
    with pytest.raises(ValueError):
        bm.w4_gemm(x, m, out=torch.zeros((2, 63)))
    with pytest.raises(ValueError):
        bm.w4_gemm(x, bm.W4Matrix(*tensors(lead=(3,))))
    g = bm.W4Matrix(*tensors(lead=(5,)))
    w = bm.W4Layer(g, g, bm.W4Matrix(*tensors(lead=(5,), N=256, K=64)))
    for xs, s in [(x, torch.zeros(2, 5)), (x, torch.zeros(3, 4)), (x.half(), torch.zeros(2, 4)),
                  (x, torch.zeros(2, 4, dtype=torch.float64)), (x, torch.zeros(2, 4))]:
        with pytest.raises(ValueError):
            bm.forward_w4(xs, s, 2, w)
