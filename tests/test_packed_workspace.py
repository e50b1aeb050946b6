"""The packed forward's workspace (no GPU): sizes that split their keys need one, and a missing, short, misaligned
or overlapping one is refused before anything is enqueued."""
import pytest

from test_packed_refusals import A, FWD, FWD_ARGS, INVALID, WORKSPACE, at, call, lib  # noqa: F401

# N, Tq, Tk, H, Hkv: few query rows against many keys
SPLIT = [(1, 1, 100000, 8, 1), (1, 1, 20011, 8, 1), (40, 40, 196000, 40, 8), (6, 6, 1557, 8, 2), (2, 20, 13097, 4, 4)]
# and sizes that fill the GPU unsplit, or have no room to split
WHOLE = [(3, 41841, 41841, 12, 12), (700, 1400, 1400, 2, 1), (1, 1, 300, 8, 8), (257, 257, 100000, 8, 1)]


@pytest.mark.parametrize("size", SPLIT)
def test_split_calls_refuse_a_bad_workspace(lib, size):  # noqa: F811
    N, Tq, Tk, H, Hkv = size
    need = lib.wan_attn_varlen_fwd_workspace_size(N, Tq, Tk, H, Hkv, 128)
    # a part's fp32 rows twice at least, and no more than K and V or 16 MB (rounded up)
    assert need >= 2 * Tq * H * 516 and need <= max(Tk * Hkv * 512, 16 << 20) + Tq * 4 + 1024
    kw = dict(N=N, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, ldq=H * 128, ldk=Hkv * 128, ldv=Hkv * 128)
    fwd = lambda **more: call(lib.wan_attn_varlen_fwd, FWD, FWD_ARGS, **kw, **more)         # noqa: E731
    assert fwd(ws=None, wsb=0) == WORKSPACE and fwd(ws=None, wsb=need) == WORKSPACE
    assert fwd(wsb=need - 1) == WORKSPACE and fwd(ws=at(A[7], 16), wsb=need) == WORKSPACE
    for other in (0, 1, 2, 3, 4, 5, 6):                                   # over q, k, v, o, lse and the offsets
        assert fwd(ws=A[other], wsb=need) == INVALID


@pytest.mark.parametrize("size", WHOLE)
def test_whole_calls_need_none(lib, size):  # noqa: F811
    assert lib.wan_attn_varlen_fwd_workspace_size(*size, 128) == 0
