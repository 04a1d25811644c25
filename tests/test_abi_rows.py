"""Refusals of the calls that move and shape rows between products and of the adapters' product, without a GPU: every
check runs on the host before any HIP call, in the C ABI and in the binding."""
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


def kinds(gmi):
    return gmi.GMI_ERR_INVALID_ARG, gmi.GMI_ERR_UNSUPPORTED, gmi.GMI_ERR_MISALIGNED


def refused(call, status, cases):
    for kw in cases:
        assert call(**kw) == status, kw


def test_group_rows_refusals(gmi):
    def call(n=5000, groups=8, index=A16, offsets=A16 * 2, order=A16 * 3, place=A16 * 4, ws=A16 * 5, nbytes=1 << 20):
        return gmi.lib().gmi_group_rows(n, groups, index, offsets, order, place, ws, nbytes, None)

    bad, uns, mis = kinds(gmi)
    refused(call, bad, [dict(n=-1), dict(groups=0), dict(index=None), dict(offsets=None), dict(order=None), dict(place=None)])
    refused(call, uns, [dict(groups=1025), dict(n=2 ** 31 - 2 ** 17), dict(n=2 ** 31 - 1)])
    refused(call, mis, [dict(index=A16 + 2), dict(offsets=A16 + 1), dict(order=A16 + 2), dict(place=A16 + 3), dict(ws=A16 + 8)])
    need = gmi.lib().gmi_group_rows_workspace_bytes(5000, 8)
    assert need > 0
    refused(call, gmi.GMI_ERR_WORKSPACE, [dict(ws=None), dict(nbytes=need - 1), dict(n=2 ** 31 - 2 ** 17 - 1, nbytes=0)])
    for n, g in ((2048, 8), (0, 8), (-1, 8), (5000, 0), (5000, 1025)):
        assert gmi.lib().gmi_group_rows_workspace_bytes(n, g) == 0


def test_permute_refusals(gmi):
    def call(T=4, k=2, K=256, dt=2, x=A16, ldx=256, xs=A16 * 2, ldxs=2, sr=A16 * 3, rows=8, out=A16 * 4, ldo=256,
             os=A16 * 5, ldos=2):
        return gmi.lib().gmi_moe_permute(T, k, K, dt, x, ldx, xs, ldxs, sr, rows, out, ldo, os, ldos, None)

    bad, uns, mis = kinds(gmi)
    refused(call, bad, [dict(T=-1), dict(k=0), dict(K=0), dict(rows=-1), dict(x=None), dict(sr=None), dict(out=None),
                        dict(xs=None), dict(os=None), dict(dt=1), dict(ldx=240), dict(ldo=128), dict(ldxs=1), dict(ldos=1)])
    refused(call, uns, [dict(k=17), dict(dt=3), dict(dt=9), dict(T=2 ** 30, k=2)])
    refused(call, mis, [dict(K=248), dict(x=A16 + 8), dict(out=A16 + 8), dict(ldx=264), dict(ldo=264), dict(sr=A16 + 2),
                        dict(xs=A16 + 2), dict(os=A16 + 2), dict(dt=1, K=252, xs=None, os=None)])
    assert call(T=0, x=None) == gmi.GMI_OK and call(rows=0, out=None) == gmi.GMI_OK


def test_unpermute_refusals(gmi):
    def call(T=4, k=2, K=256, dt=1, y=A16, ldy=256, rows=8, sr=A16 * 3, w=A16 * 4, add=A16 * 5, lda=256, out=A16 * 6,
             ldo=256):
        return gmi.lib().gmi_moe_unpermute(T, k, K, dt, y, ldy, rows, sr, w, add, lda, out, ldo, None)

    bad, uns, mis = kinds(gmi)
    refused(call, bad, [dict(T=-1), dict(k=0), dict(K=0), dict(rows=-1), dict(y=None), dict(sr=None), dict(out=None),
                        dict(ldy=248), dict(lda=8), dict(ldo=0)])
    refused(call, uns, [dict(k=17), dict(dt=2), dict(dt=3), dict(T=2 ** 30, k=2)])
    refused(call, mis, [dict(K=252), dict(y=A16 + 8), dict(out=A16 + 8), dict(add=A16 + 4), dict(ldy=260), dict(ldo=260),
                        dict(lda=260), dict(sr=A16 + 2), dict(w=A16 + 2)])
    assert call(T=0, y=None) == gmi.GMI_OK


def test_unpermute_bwd_refusals(gmi):
    def call(T=4, k=2, K=256, dt=1, d=A16, ldd=256, sr=A16 * 2, w=A16 * 3, y=A16 * 4, ldy=256, rows=8, dr=None, lddr=0,
             q=A16 * 6, ldq=256, s=A16 * 7, lds=2, dw=A16 * 8):
        return gmi.lib().gmi_moe_unpermute_bwd(T, k, K, dt, d, ldd, sr, w, y, ldy, rows, dr, lddr, q, ldq, s, lds, dw, None)

    bad, uns, mis = kinds(gmi)
    wide = dict(q=None, s=None, dr=A16 * 9, lddr=256)
    refused(call, bad, [dict(T=-1), dict(k=0), dict(K=0), dict(rows=-1), dict(d=None), dict(sr=None), dict(y=None),
                        dict(ldd=8), dict(ldy=8), dict(q=None), dict(s=None), dict(q=None, s=None, dw=None), dict(dr=A16 * 9, lddr=256),
                        dict(ldq=248), dict(lds=1), dict(wide, lddr=248)])
    refused(call, uns, [dict(k=17), dict(dt=2), dict(dt=3), dict(T=2 ** 30, k=2)])
    refused(call, mis, [dict(K=252), dict(d=A16 + 8), dict(y=A16 + 8), dict(ldd=260), dict(ldy=260), dict(q=A16 + 4),
                        dict(ldq=260), dict(s=A16 + 2), dict(sr=A16 + 1), dict(w=A16 + 2), dict(dw=A16 + 2),
                        dict(wide, dr=A16 + 8), dict(wide, lddr=260)])
    assert call(T=0, d=None) == gmi.GMI_OK


def test_swiglu_refusals(gmi):
    def fwd(rows=4, N=256, dt=1, a=A16, lda=512, live=A16 * 2, y=A16 * 3, ldy=256, q=A16 * 4, ldq=256, s=A16 * 5, lds=2):
        return gmi.lib().gmi_swiglu_quant(rows, N, dt, a, lda, live, y, ldy, q, ldq, s, lds, None)

    def bwd(rows=4, N=256, dt=1, a=A16, lda=512, live=A16 * 2, d=A16 * 3, ldd=256, da=None, ldda=0, q=A16 * 4, ldq=512,
            s=A16 * 5, lds=4):
        return gmi.lib().gmi_swiglu_bwd(rows, N, dt, d, ldd, a, lda, live, da, ldda, q, ldq, s, lds, None)

    bad, uns, mis = kinds(gmi)
    for call in (fwd, bwd):
        refused(call, bad, [dict(rows=-1), dict(N=0), dict(a=None), dict(lda=504), dict(q=None), dict(s=None), dict(ldq=248),
                            dict(lds=1)])
        refused(call, uns, [dict(dt=2), dict(dt=3), dict(N=(1 << 22) + 8)])
        refused(call, mis, [dict(N=252), dict(a=A16 + 8), dict(lda=516), dict(live=A16 + 2), dict(q=A16 + 4), dict(ldq=516),
                            dict(s=A16 + 2)])
        assert call(rows=0, a=None) == gmi.GMI_OK
    refused(fwd, bad, [dict(y=None, q=None, s=None), dict(ldy=248)])
    refused(fwd, mis, [dict(y=A16 + 8), dict(ldy=260)])
    wide = dict(q=None, s=None, da=A16 * 9, ldda=512)
    refused(bwd, bad, [dict(d=None), dict(ldd=248), dict(q=None, s=None), dict(da=A16 * 9, ldda=512), dict(wide, ldda=256),
                       dict(lds=3)])
    refused(bwd, mis, [dict(d=A16 + 8), dict(ldd=260), dict(wide, da=A16 + 8), dict(wide, ldda=516)])


def test_lora_refusals(gmi):
    def call(M=100, N=256, K=512, rank=16, L=4, dt=1, X=A16, ldx=512, A=A16 * 2, lda=512, sa=8192, B=A16 * 3, ldb=16,
             sb=4096, s=A16 * 4, index=A16 * 5, order=A16 * 6, base=A16 * 7, ldbase=256, Y=A16 * 8, ldy=256, ws=A16 * 64,
             nbytes=1 << 30):
        return gmi.lib().gmi_gemm_lora(M, N, K, rank, L, dt, X, ldx, A, lda, sa, B, ldb, sb, s, index, order, base, ldbase,
                                       Y, ldy, ws, nbytes, None)

    bad, uns, mis = kinds(gmi)
    refused(call, bad, [dict(M=-1), dict(N=-8), dict(K=0), dict(rank=0), dict(L=-1), dict(X=None), dict(A=None), dict(B=None),
                        dict(index=None), dict(Y=None), dict(ldx=504), dict(lda=504), dict(ldb=8), dict(ldbase=248),
                        dict(ldy=248), dict(sa=8184), dict(sb=4088), dict(sa=-8192), dict(base=A16 * 8, ldbase=264)])
    refused(call, uns, [dict(dt=2), dict(dt=3), dict(rank=136), dict(M=(1 << 29) + 1), dict(N=2 ** 31 - 8, ldy=2 ** 31 - 8),
                        dict(K=2 ** 31 - 8)])
    # more workgroups than a launch holds; ends of parts past 32 bits
    refused(call, uns, [dict(M=(1 << 26) + 1), dict(N=2 ** 31 - 2 ** 18, ldy=2 ** 31), dict(K=2 ** 31 - 2 ** 18)])
    refused(call, mis, [dict(N=252), dict(K=508), dict(rank=12), dict(X=A16 + 8), dict(A=A16 + 8), dict(B=A16 + 8),
                        dict(base=A16 + 8), dict(Y=A16 + 8), dict(ldx=516), dict(lda=516), dict(ldb=20), dict(ldbase=260),
                        dict(ldy=260), dict(sa=8196), dict(sb=4100), dict(s=A16 + 2), dict(index=A16 + 2), dict(order=A16 + 2),
                        dict(ws=A16 + 8)])
    need = gmi.lib().gmi_gemm_lora_workspace_bytes(100, 256, 512, 16)
    assert need >= 100 * 16 * 4
    refused(call, gmi.GMI_ERR_WORKSPACE, [dict(ws=None), dict(nbytes=need - 1)])
    assert call(M=0, X=None) == gmi.GMI_OK and call(N=0, Y=None) == gmi.GMI_OK
    for M, N, K, r in ((0, 8, 8, 8), (8, 0, 8, 8), (8, 8, 0, 8), (8, 8, 8, 0), (8, 8, 8, 136), ((1 << 29) + 1, 8, 8, 8)):
        assert gmi.lib().gmi_gemm_lora_workspace_bytes(M, N, K, r) == 0


def test_binding_refuses_wrong_tensors(gmi):
    # host tensors, wrong types and shapes never reach the library
    bf, i32 = torch.bfloat16, torch.int32
    x, slots = torch.zeros(4, 256, dtype=bf), torch.zeros(4, 2, dtype=i32)
    ws = torch.empty(1 << 16, dtype=torch.uint8)

    def no(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)

    no("contiguous device tensor", gmi.group_rows, slots, 4)
    no("float16 or bfloat16", gmi.moe_permute, x.float(), slots)
    no("device", gmi.moe_permute, x, slots)
    no("two dimensions", gmi.moe_unpermute, x[0], slots, out=x)
    no("device", gmi.moe_unpermute, x, slots)
    no("device", gmi.moe_unpermute_bwd, x, slots)
    no("rows of the forward", gmi.moe_unpermute_bwd, x, slots, dweights=torch.zeros(4, 2))
    no("quantize=True", gmi.moe_unpermute_bwd, x, slots, scales=torch.zeros(8, 2))
    no("row_grad=True", gmi.moe_unpermute_bwd, x, slots, rows=x, drows=x, row_grad=False)
    no("rows of the forward", gmi.moe_unpermute_bwd, x, slots, row_grad=False)
    no("device", gmi.swiglu_quant, x)
    no("quantize=True", gmi.swiglu_quant, x, q=x, quantize=False)
    no("device", gmi.swiglu_bwd, x[:, :128], x)
    no("quantize=True", gmi.swiglu_bwd, x[:, :128], x, scales=torch.zeros(4, 2))
    A, B = torch.zeros(3, 16, 256, dtype=bf), torch.zeros(3, 64, 16, dtype=bf)
    no("device", gmi.gemm_lora, x, A, B, slots[:, 0], workspace=ws)
    native = gmi._bound()
    for name, n in (("group_rows", 7), ("moe_permute", 6), ("moe_unpermute", 6), ("moe_unpermute_bwd", 9),
                    ("swiglu_quant", 6), ("swiglu_bwd", 7), ("gemm_lora", 10)):
        with pytest.raises(TypeError, match=f"{n} arguments"):
            getattr(native, name)(x)
        with pytest.raises(ValueError, match="must be a tensor"):
            getattr(native, name)(*([1.0] * n))
    with pytest.raises(TypeError, match="7 addresses"):
        native.bind_rows(1, 2)
    with pytest.raises(ValueError, match="NULL"):
        native.bind_rows(1, 2, 3, 4, 5, 6, 0, len)


def test_stream_of_another_device_is_refused(gmi, monkeypatch):
    class Stream:
        cuda_stream, device_index = 7, 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 40 + d, raising=False)
    assert gmi._stream_on(None, 0) == 40 and gmi._stream_on(9, 0) == 9
    with pytest.raises(ValueError, match="current"):
        gmi._stream_on(None, 1)
    with pytest.raises(ValueError, match="stream"):
        gmi._stream_on(Stream(), 0)
    Stream.device_index = 0
    assert gmi._stream_on(Stream(), 0) == 7
