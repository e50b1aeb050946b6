"""What the packed attention and int8 calls refuse, on the host, before anything is enqueued (no GPU)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5
A = [ctypes.c_void_p(0x100000 + i * 0x10000000) for i in range(14)]     # never dereferenced on these paths


def at(p, off):
    return ctypes.c_void_p(p.value + off)


@pytest.fixture()
def lib(built):
    from video_dit_full_b200 import wan_attn
    return wan_attn.lib()


def call(fn, names, defaults, **kw):
    assert not set(kw) - set(names)
    return fn(*[kw.get(n, d) for n, d in zip(names, defaults)])


FWD = ("q", "k", "v", "o", "lse", "cu_q", "cu_k", "N", "Tq", "Tk", "H", "Hkv", "D", "ldq", "ldk", "ldv", "causal", "ws",
       "wsb", "st")
FWD_ARGS = (*A[:7], 2, 300, 400, 4, 2, 128, 512, 256, 256, 1, A[7], 1 << 27, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID),
    (dict(cu_q=None), INVALID), (dict(cu_k=at(A[6], 2)), INVALID), (dict(N=0), INVALID), (dict(Tq=-1), INVALID),
    (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID), (dict(D=64), UNSUPPORTED),
    (dict(ldq=504), INVALID), (dict(ldk=260), INVALID), (dict(ldv=128), INVALID), (dict(q=at(A[0], 8)), INVALID),
    (dict(o=A[0]), INVALID), (dict(o=A[1]), INVALID), (dict(lse=A[3]), INVALID), (dict(lse=A[5]), INVALID),
    (dict(o=at(A[0], 512), ldq=1024), INVALID),
    (dict(Tq=1 << 30, H=65536, Hkv=1, ldq=65536 * 128), INVALID), (dict(Tk=0x7fffffff), INVALID),
    (dict(N=1 << 24, H=64, Hkv=2), INVALID)])
def test_packed_forward(lib, kw, want):
    assert call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, **kw) == want


def test_packed_forward_workspace(lib):
    size = lib.wan_attn_varlen_fwd_workspace_size
    assert size(1, 1, 1 << 20, 8, 4, 96) == 0 and size(0, 1, 1, 1, 1, 128) == 0
    need = size(1, 1, 100000, 8, 1, 128)                 # one token, many keys: split
    kw = dict(N=1, Tq=1, Tk=100000, H=8, Hkv=1, ldq=1024, ldk=128, ldv=128)
    if need:
        assert call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, **kw, ws=None, wsb=0) == WORKSPACE
        assert call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, **kw, wsb=need - 1) == WORKSPACE
        assert call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, **kw, ws=at(A[7], 16)) == WORKSPACE
        assert call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, **kw, ws=A[1]) == INVALID
    # nothing to do: no launch, no GPU
    assert call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, Tq=0, q=None, o=None, lse=None) == 0


BWD = ("q", "k", "v", "o", "do", "lse", "dq", "dk", "dv", "cu_q", "cu_k", "N", "Tq", "Tk", "H", "Hkv", "D", "ldq", "ldk",
       "ldv", "lddq", "lddk", "lddv", "causal", "ws", "wsb", "st")
BWD_ARGS = (*A[:11], 2, 300, 400, 4, 2, 128, 512, 256, 256, 512, 256, 256, 1, A[11], 1 << 27, None)


@pytest.mark.parametrize("kw,want", [
    (dict(do=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID), (dict(lse=None), INVALID),
    (dict(D=256), UNSUPPORTED), (dict(Hkv=3), INVALID), (dict(lddk=64), INVALID), (dict(lddq=516), INVALID),
    (dict(dq=A[0]), INVALID), (dict(dk=A[8]), INVALID), (dict(dv=A[4]), INVALID), (dict(dk=A[9]), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=0), WORKSPACE), (dict(ws=at(A[11], 128)), WORKSPACE), (dict(ws=A[2]), INVALID),
    # slices of one buffer: too close, and another stride
    (dict(dq=A[6], dk=at(A[6], 512), lddq=1024, lddk=1024, Tk=300), INVALID),
    (dict(dq=A[6], dk=at(A[6], 1024), lddq=1024, lddk=512, Tk=300), INVALID)])
def test_packed_backward(lib, kw, want):
    assert call(lib.wan_attn_varlen_bwd, BWD, BWD_ARGS, **kw) == want


def test_packed_sizes(lib):
    size = lib.wan_attn_varlen_bwd_workspace_size
    assert size(2, 300, 400, 4, 3, 128) == 0 and size(2, 300, 400, 4, 2, 64) == 0 and size(2, -1, 4, 4, 2, 128) == 0
    assert size(2, 300, 400, 4, 2, 128) > 0


X, W, S, B, Y, C = A[:6]


def test_int8_calls(lib):
    p = 0x10000000                                       # the pointers' distance
    rows = lib.wan_int8_quantize_rows
    assert rows(X, C, S, 10, 24, 24, None) == INVALID                     # K % 16
    assert rows(X, C, S, 10, 32, 24, None) == INVALID                     # rows overlap
    assert rows(X, C, S, 10, 32, 36, None) == INVALID                     # row stride % 8
    assert rows(X, X, S, 10, 32, 32, None) == INVALID                     # codes over x
    assert rows(X, C, S, -1, 32, 32, None) == INVALID
    assert rows(X, C, S, 2, 131088, 131088, None) == INVALID              # past the sums' range
    assert rows(at(X, 8), C, S, 10, 32, 32, None) == INVALID
    assert rows(None, None, None, 0, 32, 32, None) == 0                   # no rows: nothing to do
    back = lib.wan_int8_dequantize_rows
    assert back(C, S, C, 10, 32, None) == INVALID and back(C, None, X, 10, 32, None) == INVALID
    assert back(None, None, None, 0, 32, None) == 0
    gemm = lib.wan_int8_gemm
    assert gemm(C, S, W, B, None, Y, 10, 20, 32, None) == INVALID         # N % 8
    assert gemm(C, S, W, B, None, None, 10, 24, 32, None) == INVALID
    assert gemm(C, S, W, B, at(X, 4), Y, 10, 24, 32, None) == INVALID     # bias alignment
    assert gemm(C, S, W, B, None, C, 10, 24, 32, None) == INVALID         # y over the codes
    assert gemm(C, at(S, 2), W, B, None, Y, 10, 24, 32, None) == INVALID
    assert gemm(C, S, W, B, at(Y, 16), Y, 10, 24, 32, None) == INVALID    # bias inside y
    assert gemm(None, None, None, None, None, None, 0, 24, 32, None) == 0
    linear = lib.wan_int8_linear
    assert linear(X, W, B, None, Y, C, at(C, 64), 10, 24, 32, 32, None) == INVALID    # scales inside the codes
    assert linear(X, W, B, None, Y, W, S, 10, 24, 32, 32, None) == INVALID            # codes over the weight's
    assert linear(X, W, B, None, Y, C, S, 10, 24, 32, 16, None) == INVALID
    assert linear(None, None, None, None, None, None, None, 0, 24, 32, 32, None) == 0
    for grad in (lib.wan_int8_grad_weight, lib.wan_int8_grad_input):
        assert grad(X, C, S, X, 10, 24, 32, None) == INVALID
        assert grad(None, C, S, Y, 10, 24, 32, None) == INVALID
        assert grad(X, C, S, Y, 10, 23, 32, None) == INVALID
        assert grad(X, at(C, 1), S, Y, 10, 24, 32, None) == INVALID
    assert lib.wan_int8_grad_weight(None, None, None, at(Y, 4), 0, 24, 32, None) == INVALID
    assert p


def test_int8_sizes_near_2_31(lib):
    """Rounding such a size up to a tile would pass 32 bits."""
    far = [ctypes.c_void_p(0x1000000000000 + i * 0x10000000000) for i in range(5)]
    m = 0x7fffffff
    assert lib.wan_int8_quantize_rows(*far[:3], m, 16, 16, None) == INVALID
    assert lib.wan_int8_dequantize_rows(*far[:3], m, 16, None) == INVALID
    assert lib.wan_int8_gemm(far[0], far[1], far[2], far[3], None, far[4], m, 8, 16, None) == INVALID
    assert lib.wan_int8_gemm(far[0], far[1], far[2], far[3], None, far[4], 8, 0x7ffffff8, 16, None) == INVALID
    assert lib.wan_int8_grad_weight(*far[:4], 8, 0x7ffffff8, 16, None) == INVALID
    assert lib.wan_int8_grad_input(*far[:4], m, 8, 16, None) == INVALID


def test_python_refuses_what_is_not_on_the_gpu(built):
    import torch
    import video_dit_full_b200 as wa
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(TypeError):
        wa.varlen_fwd(q, q, q, cu, cu)
    with pytest.raises(TypeError):
        wa.int8_quantize_rows(torch.zeros(4, 32, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        wa.int8_linear(torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.int8), torch.ones(8))
    with pytest.raises(TypeError):
        wa.int8_grad_weight(torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 32, dtype=torch.int8), torch.ones(4))
