"""Refusals of the 8-bit operators' C entries: each is returned before anything is enqueued
(no GPU needed; the addresses are never followed), and the workspace sizes."""
import ctypes

import pytest

OK, EINVAL, ENOSPC, EUNSUPPORTED = 0, 1, 2, 3
A = 4096  # a non-null address


def L():
    import token_routing_grouped_amd as moe
    return moe.lib()


def meta(N=4, K=2, E=3, cap=8, p=A):
    from token_routing_grouped_amd._binding import _CMeta
    return ctypes.byref(_CMeta(N, K, E, cap, *([p] * 8)))


def test_quantize_rows_refusals():
    f = L().moe_quantize_rows
    assert f(None, 0, 64, 0, None, None, 0, None) == OK  # no rows: nothing to do
    assert f(A, -1, 64, 0, A, A, 0, None) == EINVAL
    for H in (0, -8, 12, (1 << 20) + 8):
        assert f(A, 1, H, 0, A, A, 0, None) == EUNSUPPORTED
    assert f(A, 1, 64, 2, A, A, 0, None) == EUNSUPPORTED
    assert f(A, 1, 64, 0, A, A, 2, None) == EUNSUPPORTED
    assert f(A, 1 << 28, 128, 0, A, A, 0, None) == EUNSUPPORTED  # more lanes than a launch
    for x, q, s in ((None, A, A), (A, None, A), (A, A, None)):
        assert f(x, 1, 64, 0, q, s, 0, None) == EINVAL


def test_quantize_weights_refusals():
    f = L().moe_quantize_weights
    assert f(A, 0, 64, 64, 0, A, A, 0, None) == EINVAL
    assert f(A, 1025, 64, 64, 0, A, A, 0, None) == EINVAL
    for K, C in ((8, 64), (64, 24), (0, 64), ((1 << 20) + 16, 64), (64, (1 << 21) + 16)):
        assert f(A, 1, K, C, 0, A, A, 0, None) == EUNSUPPORTED
    assert f(A, 1, 64, 64, 3, A, A, 0, None) == EUNSUPPORTED
    assert f(A, 1, 64, 64, 0, A, A, -1, None) == EUNSUPPORTED
    assert f(A, 1024, 1 << 20, 1 << 21, 0, A, A, 0, None) == EUNSUPPORTED
    for w, q, s in ((None, A, A), (A, None, A), (A, A, None)):
        assert f(w, 1, 64, 64, 0, q, s, 0, None) == EINVAL


def test_rmsnorm_refusals():
    f = L().moe_rmsnorm_forward

    def call(x=A, res=None, w=A, eps=1e-6, N=2, H=64, dt=0, ro=None, y=A, q=None, s=None, st=0):
        return f(x, res, w, eps, N, H, dt, ro, y, q, s, st, None, None)

    assert call(N=0, x=None, w=None, y=None) == OK
    assert call(N=-1) == EINVAL
    assert call(eps=-1.0) == EINVAL and call(eps=float("nan")) == EINVAL
    assert call(H=20) == EUNSUPPORTED and call(H=(1 << 20) + 8) == EUNSUPPORTED
    assert call(dt=2) == EUNSUPPORTED
    assert call(x=None) == EINVAL and call(w=None) == EINVAL
    assert call(y=None) == EINVAL                      # no output
    assert call(q=A) == EINVAL and call(s=A) == EINVAL  # 8 bits need both
    assert call(q=A, s=A, st=5) == EUNSUPPORTED
    assert call(res=A) == EINVAL and call(ro=A) == EINVAL  # a residual and its output


def test_rmsnorm_backward_refusals():
    f, ws = L().moe_rmsnorm_backward, L().moe_rmsnorm_backward_workspace
    need = ws(100, 64)
    assert need == 100 * 64 * 4 and ws(0, 64) == 0 and ws(1 << 20, 64) == 512 * 64 * 4

    def call(dy=A, r=A, w=A, rstd=A, N=100, H=64, dt=0, dx=A, dw=A, wk=A, nb=need):
        return f(dy, r, w, rstd, None, N, H, dt, dx, dw, wk, nb, None)

    assert call(N=-1) == EINVAL
    assert call(H=12) == EUNSUPPORTED and call(dt=9) == EUNSUPPORTED
    for k in ("dy", "r", "w", "rstd", "dx", "dw"):
        assert call(**{k: None}) == EINVAL
    assert call(nb=need - 1) == ENOSPC and call(wk=None) == ENOSPC


def test_grouped_product_refusals():
    f = L().moe_grouped_gemm_fp8

    def call(m=None, a=A, sa=A, ta=0, w=A, sw=A, tw=0, K=64, C=64, out=A):
        return f(meta() if m is None else m, a, sa, ta, w, sw, tw, K, C, 1, out, None)

    assert f(None, A, A, 0, A, A, 0, 64, 64, 1, A, None) == EINVAL
    assert call(m=meta(K=0)) == EINVAL
    for K, C in ((8, 64), (64, 8), ((1 << 20) + 16, 64), (64, (1 << 21) + 16), (-16, 64)):
        assert call(K=K, C=C) == EUNSUPPORTED
    assert call(ta=2) == EUNSUPPORTED and call(tw=2) == EUNSUPPORTED
    for k in ("a", "sa", "w", "sw", "out"):
        assert call(**{k: None}) == EINVAL
    assert call(m=meta(N=0), a=None, out=None) == OK
    assert call(m=meta(cap=0), a=None, out=None) == OK
    # more tiles than one launch holds
    assert call(m=meta(N=1 << 26, K=8, cap=1 << 29), C=1 << 21) == EUNSUPPORTED


def test_expert_forward_refusals():
    f, ws = L().moe_expert_forward_fp8, L().moe_expert_forward_fp8_workspace
    need = ws(meta(), 64, 32)
    assert need == 256 + 256 + 8 * 64 * 4 + 8 * 32 * 4
    assert ws(meta(cap=61), 64, 32) == 2048 + 256 + 15616 + 7936  # few tiles of 32 rows
    n = 1 << 16  # neither few rows per expert nor few tiles
    assert ws(meta(cap=n), 64, 32) == n * 32 + n + n * 64 * 2 + n

    def call(m=None, x=A, xs=A, tx=0, u=A, us=A, d=A, ds=A, tw=0, H=64, I=32, lay=0, out=A, wk=A, nb=need):
        return f(meta() if m is None else m, x, xs, tx, u, us, d, ds, tw, H, I, lay, None, out, wk, nb, None)

    assert f(None, A, A, 0, A, A, A, A, 0, 64, 32, 0, None, A, A, 1 << 20, None) == EINVAL
    for H, I in ((24, 32), (64, 24), (0, 32), ((1 << 20) + 16, 32), (64, (1 << 20) + 16)):
        assert call(H=H, I=I) == EUNSUPPORTED
    assert call(tx=2) == EUNSUPPORTED and call(tw=-1) == EUNSUPPORTED and call(lay=2) == EUNSUPPORTED
    for k in ("x", "xs", "u", "us", "d", "ds", "out"):
        assert call(**{k: None}) == EINVAL
    assert call(nb=need - 1) == ENOSPC and call(wk=None) == ENOSPC
    assert call(m=meta(N=0), x=None, out=None) == OK


def test_refusals_of_addresses():
    """16 bytes for what is read and written in pieces of 16, 8 for q of rows, 4 for fp32 scales
    and rstd; e8m0 scales anywhere."""
    l = L()
    B, R, Z = A + 8, A + 4, A + 2
    assert l.moe_quantize_rows(B, 1, 64, 0, A, A, 0, None) == EINVAL
    assert l.moe_quantize_rows(A, 1, 64, 0, R, A, 0, None) == EINVAL
    assert l.moe_quantize_rows(A, 1, 64, 0, A, Z, 0, None) == EINVAL
    for w, q, s in ((B, A, A), (A, B, A), (A, A, Z)):
        assert l.moe_quantize_weights(w, 1, 64, 64, 0, q, s, 0, None) == EINVAL
    ok = [A, A, A, 1e-6, 1, 64, 0, A, A, A, A, 0, A, None]
    for i, v in ((0, B), (1, B), (2, B), (7, B), (8, B), (9, R), (10, Z), (12, Z)):
        assert l.moe_rmsnorm_forward(*ok[:i], v, *ok[i + 1:]) == EINVAL
    ok = [A, A, A, A, A, 1, 64, 0, A, A, A, 1 << 20, None]
    for i, v in ((0, B), (1, B), (2, B), (3, Z), (4, B), (8, B), (9, B), (10, B)):
        assert l.moe_rmsnorm_backward(*ok[:i], v, *ok[i + 1:]) == EINVAL
    ok = [meta(), A, A, 0, A, A, 0, 64, 64, 1, A, None]
    for i, v in ((1, B), (2, Z), (4, B), (5, Z), (10, B)):
        assert l.moe_grouped_gemm_fp8(*ok[:i], v, *ok[i + 1:]) == EINVAL
    ok = [meta(), A, A, 0, A, A, A, A, 0, 64, 32, 0, A, A, A, 1 << 20, None]
    for i, v in ((1, B), (2, Z), (4, B), (5, Z), (6, B), (7, Z), (12, B), (13, B), (14, B)):
        assert l.moe_expert_forward_fp8(*ok[:i], v, *ok[i + 1:]) == EINVAL


def test_binding_refuses_host_tensors():
    import torch
    import token_routing_grouped_amd as moe
    x = torch.zeros(2, 64)
    with pytest.raises(TypeError, match="device tensor"):
        moe.moe_quantize_rows(x, x, x)
    with pytest.raises(TypeError, match="device tensor"):
        moe.moe_rmsnorm_forward(x, x[0])
