"""Refusals of the block-scaled fp8 mixture-of-experts calls, without a GPU:
every check runs on the host before any HIP call, in the C ABI and in the
binding."""
import pytest
import torch

A16 = 0x10000  # fake, 16-byte aligned device addresses: never dereferenced by a rejected call


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    if not g.LIB_PATH.exists():
        from grouped_mixed_input_amd import build

        build.build()
    g.lib()
    return g


def _norm(gmi, rows=4, K=256, x=A16, ldx=256, res=A16 * 2, ldr=256, w=A16 * 3, eps=1e-6, dt=1, h=A16 * 4, ldh=256,
          y=None, ldy=0, q=A16 * 5, ldq=256, s=A16 * 6, lds=2):
    return gmi.lib().gmi_rmsnorm_quant(rows, K, x, ldx, res, ldr, w, eps, dt, h, ldh, y, ldy, q, ldq, s, lds, None)


def test_rmsnorm_quant_refusals(gmi):
    bad, mis, uns = gmi.GMI_ERR_INVALID_ARG, gmi.GMI_ERR_MISALIGNED, gmi.GMI_ERR_UNSUPPORTED
    for kw in (dict(rows=-1), dict(K=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
               dict(w=None), dict(ldx=248), dict(ldr=128), dict(ldh=0), dict(q=None), dict(s=None),
               dict(q=None, s=None), dict(ldq=248), dict(lds=1), dict(y=A16 * 7, ldy=100)):
        assert _norm(gmi, **kw) == bad, kw
    for kw in (dict(K=252), dict(x=A16 + 8), dict(ldx=260), dict(res=A16 + 4), dict(w=A16 + 2), dict(h=A16 + 8),
               dict(ldh=257), dict(q=A16 + 4), dict(ldq=260), dict(s=A16 + 2), dict(y=A16 + 2, ldy=256)):
        assert _norm(gmi, **kw) == mis, kw
    for kw in (dict(dt=2), dict(dt=3), dict(dt=7), dict(K=32776, ldx=32776, ldr=32776, ldh=32776, ldq=32776, lds=300)):
        assert _norm(gmi, **kw) == uns, kw
    assert _norm(gmi, rows=0, x=None, w=None) == gmi.GMI_OK
    assert "rmsnorm_quant" in (_norm(gmi, K=0), gmi.lib().gmi_last_error().decode())[1]


def _bwd(gmi, rows=4, K=256, dy=A16, lddy=256, h=A16 * 2, ldh=256, w=A16 * 3, dres=A16 * 4, lddr=256, eps=1e-6, dt=0,
         dh=A16 * 5, lddh=256, dw=A16 * 6, ws=A16 * 64, ws_bytes=64):
    return gmi.lib().gmi_rmsnorm_bwd(rows, K, dy, lddy, h, ldh, w, dres, lddr, eps, dt, dh, lddh, dw, ws, ws_bytes,
                                     None)


def test_rmsnorm_bwd_refusals(gmi):
    bad, mis, uns = gmi.GMI_ERR_INVALID_ARG, gmi.GMI_ERR_MISALIGNED, gmi.GMI_ERR_UNSUPPORTED
    for kw in (dict(rows=-1), dict(K=0), dict(eps=-1.0), dict(dy=None), dict(h=None), dict(w=None), dict(dh=None),
               dict(lddy=8), dict(ldh=8), dict(lddr=8), dict(lddh=8)):
        assert _bwd(gmi, **kw) == bad, kw
    for kw in (dict(K=250), dict(dy=A16 + 8), dict(lddr=260), dict(dw=A16 + 2), dict(dh=A16 + 8)):
        assert _bwd(gmi, **kw) == mis, kw
    assert _bwd(gmi, dt=3) == uns
    assert _bwd(gmi, ws_bytes=63) == gmi.GMI_ERR_WORKSPACE
    assert _bwd(gmi, ws=None, ws_bytes=1 << 20) == gmi.GMI_ERR_WORKSPACE
    assert _bwd(gmi, ws=A16 + 4, ws_bytes=1 << 20) == mis
    assert _bwd(gmi, rows=0, dw=None, ws=None) == gmi.GMI_OK
    assert gmi.lib().gmi_rmsnorm_bwd_workspace_bytes(0, 256) == 0
    assert gmi.lib().gmi_rmsnorm_bwd_workspace_bytes(8, 256) >= 256 * 4


def _f8(gmi, M=64, N=256, K=256, X=A16, ldx=256, xs=A16 * 2, ldxs=2, W=A16 * 3, ldw=256, ws=A16 * 4, ldws=2, Y=A16 * 5,
        ldy=256, work=None, nbytes=0):
    return gmi.lib().gmi_gemm_f8_block(M, N, K, X, ldx, xs, ldxs, W, ldw, ws, ldws, Y, ldy, work, nbytes, None)


def _f8g(gmi, count=4, off=A16 * 7, rows=64, N=256, K=256, X=A16, ldx=256, xs=A16 * 2, ldxs=2, W=A16 * 3, ldw=256,
         w_stride=65536, ws=A16 * 4, ldws=2, ws_stride=4, Y=A16 * 5, ldy=256, work=A16 * 64, nbytes=1 << 20):
    return gmi.lib().gmi_gemm_f8_block_grouped(count, off, rows, N, K, X, ldx, xs, ldxs, W, ldw, w_stride, ws, ldws,
                                               ws_stride, Y, ldy, work, nbytes, None)


@pytest.mark.parametrize("call", [_f8, _f8g])
def test_f8_block_refusals(gmi, call):
    rows = "M" if call is _f8 else "rows"
    bad, mis, uns = gmi.GMI_ERR_INVALID_ARG, gmi.GMI_ERR_MISALIGNED, gmi.GMI_ERR_UNSUPPORTED
    for kw in ({rows: -1}, dict(N=-1), dict(K=-16), dict(X=None), dict(xs=None), dict(W=None), dict(ws=None),
               dict(Y=None), dict(ldx=240), dict(ldw=128), dict(ldxs=1), dict(ldws=1), dict(ldy=248)):
        assert call(gmi, **kw) == bad, kw
    for kw in (dict(K=248), dict(ldx=264), dict(ldw=264), dict(ldx=1 << 23), dict(ldy=1 << 23)):
        assert call(gmi, **kw) == uns, kw
    for kw in (dict(X=A16 + 8), dict(W=A16 + 4), dict(Y=A16 + 8), dict(ldy=260), dict(xs=A16 + 2), dict(ws=A16 + 1),
               dict(work=A16 + 8, nbytes=1 << 20)):
        assert call(gmi, **kw) == mis, kw
    for kw in ({rows: 0}, dict(N=0)):
        assert call(gmi, X=None, W=None, Y=None, xs=None, ws=None, **kw) == gmi.GMI_OK


def test_f8_block_grouped_refusals(gmi):
    bad = gmi.GMI_ERR_INVALID_ARG
    for kw in (dict(count=-1), dict(off=None), dict(w_stride=-16), dict(ws_stride=-1), dict(w_stride=65520),
               dict(ws_stride=3)):
        assert _f8g(gmi, **kw) == bad, kw
    assert _f8g(gmi, count=1025) == gmi.GMI_ERR_UNSUPPORTED
    assert _f8g(gmi, off=A16 + 2) == gmi.GMI_ERR_MISALIGNED
    assert _f8g(gmi, w_stride=65544) == gmi.GMI_ERR_MISALIGNED
    need = gmi.lib().gmi_gemm_f8_block_grouped_workspace_bytes(4)
    assert need > 0 and _f8g(gmi, nbytes=need - 1) == gmi.GMI_ERR_WORKSPACE
    assert _f8g(gmi, work=None) == gmi.GMI_ERR_WORKSPACE
    assert _f8g(gmi, count=0, off=None) == gmi.GMI_OK
    assert gmi.lib().gmi_gemm_f8_block_grouped_workspace_bytes(0) == 0
    assert gmi.lib().gmi_gemm_f8_block_grouped_workspace_bytes(2000) == 0


def _route(gmi, T=100, E=16, k=2, x=A16, ld=16, dt=3, mask=None, outs=None, ws=A16 * 64, nbytes=1 << 20):
    outs = outs or [A16 * (2 + i) for i in range(8)]
    return gmi.lib().gmi_moe_route(T, E, k, x, ld, dt, mask, 1, *outs, ws, nbytes, None)


def test_route_refusals(gmi):
    bad, mis, uns = gmi.GMI_ERR_INVALID_ARG, gmi.GMI_ERR_MISALIGNED, gmi.GMI_ERR_UNSUPPORTED
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(k=17, E=16), dict(x=None), dict(ld=15)):
        assert _route(gmi, **kw) == bad, kw
    for i in range(8):
        outs = [A16 * (2 + j) for j in range(8)]
        outs[i] = None
        assert _route(gmi, outs=outs) == bad, i
        outs[i] = A16 + 2
        assert _route(gmi, outs=outs) == mis, i
    for kw in (dict(E=1025, ld=1025), dict(k=17, E=32, ld=32), dict(dt=2), dict(dt=5), dict(T=1 << 30, k=2)):
        assert _route(gmi, **kw) == uns, kw
    assert _route(gmi, x=A16 + 2) == mis and _route(gmi, x=A16 + 1, dt=0) == mis
    need = gmi.lib().gmi_moe_route_workspace_bytes(100, 16)
    assert need > 0 and _route(gmi, nbytes=need - 1) == gmi.GMI_ERR_WORKSPACE
    assert _route(gmi, ws=None) == gmi.GMI_ERR_WORKSPACE and _route(gmi, ws=A16 + 2) == mis
    assert gmi.lib().gmi_moe_route_workspace_bytes(64, 16) == 0
    assert gmi.lib().gmi_moe_route_workspace_bytes(-1, 16) == 0


def test_route_bwd_refusals(gmi):
    def call(T=100, E=16, k=2, x=A16, ld=16, dt=3, ins=None, d=A16 * 30, ldd=16):
        ins = ins or [A16 * (2 + i) for i in range(6)]
        return gmi.lib().gmi_moe_route_bwd(T, E, k, x, ld, dt, None, 1, *ins, d, ldd, None)

    bad, mis = gmi.GMI_ERR_INVALID_ARG, gmi.GMI_ERR_MISALIGNED
    for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(x=None), dict(ld=8), dict(ldd=8), dict(d=None)):
        assert call(**kw) == bad, kw
    for i in range(6):
        ins = [A16 * (2 + j) for j in range(6)]
        ins[i] = None
        assert call(ins=ins) == bad, i
        ins[i] = A16 + 2
        assert call(ins=ins) == mis, i
    assert call(d=A16 + 2) == mis and call(dt=2) == gmi.GMI_ERR_UNSUPPORTED
    assert call(T=0, x=None) == gmi.GMI_OK


def test_binding_refuses_wrong_tensors(gmi):
    # host tensors, wrong types and shapes never reach the library
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        gmi.rmsnorm_quant(x, w)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        gmi.rmsnorm_quant(x.float(), w)
    with pytest.raises(ValueError, match="device"):
        gmi.rmsnorm_bwd(x, x, w, workspace=torch.empty(1 << 16, dtype=torch.uint8))
    f8 = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="device"):
        gmi.gemm_f8_block(f8, torch.ones(4, 2), f8, torch.ones(1, 2))
    with pytest.raises(ValueError, match="groups"):
        gmi.gemm_f8_block_grouped(torch.zeros(2, dtype=torch.int32), f8, torch.ones(4, 2), f8, torch.ones(1, 2))
    with pytest.raises(ValueError, match="logits"):
        gmi.moe_route(torch.zeros(4, 8, dtype=torch.float64), 2)
    with pytest.raises(ValueError, match="device"):
        gmi.moe_route(torch.zeros(4, 8), 2)


def test_native_marshalling_refuses_what_is_no_tensor(gmi):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be a tensor"):
        gmi._bound().rmsnorm_quant([1.0], x[0], None, 1e-6, None, None, None, None, 0)
    with pytest.raises(ValueError, match=r"\[rows\]\[K\]"):
        gmi._bound().rmsnorm_quant(x[0], x[0], None, 1e-6, None, None, None, None, 0)
    with pytest.raises(TypeError, match="9 arguments"):
        gmi._bound().rmsnorm_quant(x)
    with pytest.raises(TypeError, match="6 addresses"):
        gmi._bound().bind(1, 2)
    with pytest.raises(ValueError, match="NULL"):
        gmi._bound().bind(1, 2, 3, 4, 5, 0, len)
    with pytest.raises(ValueError, match="2\\^31|device"):
        gmi.moe_route(x.float(), 2, out=gmi.Routing(*([x] * 8)), workspace=x)


def test_empty_group_list_is_a_no_op(gmi):
    f8 = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    Y = torch.full((4, 128), 3.0, dtype=torch.bfloat16)
    got = gmi.gemm_f8_block_grouped(torch.zeros(1, dtype=torch.int32), f8, torch.ones(4, 2), f8.new_zeros(0, 128, 256),
                                    torch.ones(0, 1, 2), Y=Y)
    assert got is Y and (Y == 3.0).all()


def test_route_token_limit(gmi):
    # token numbers stay 32-bit with room for a workgroup's share past the last one
    assert _route(gmi, T=2 ** 31 - 2 ** 17, k=1) == gmi.GMI_ERR_UNSUPPORTED
    assert _route(gmi, T=2 ** 31 - 1, k=1) == gmi.GMI_ERR_UNSUPPORTED
    assert _route(gmi, T=2 ** 31 - 2 ** 17 - 1, k=1, ws=None) == gmi.GMI_ERR_WORKSPACE
