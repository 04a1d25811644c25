"""Outputs in the place of an input, without a GPU: with another leading dimension rows would be written over rows still to
be read, so every call that allows the one refuses the other, before any HIP call."""
import pytest

A16 = 0x10000  # fake, 16-byte aligned device addresses: never dereferenced by a rejected call


@pytest.fixture(scope="module")
def gmi():
    import grouped_mixed_input_amd as g

    if not g.LIB_PATH.exists():
        from grouped_mixed_input_amd import build

        build.build()
    g.lib()
    return g


@pytest.mark.parametrize("lda,ldo", [(256, 264), (512, 256)])
def test_sum_over_its_addend(gmi, lda, ldo):
    def call(T):
        return gmi.lib().gmi_moe_unpermute(T, 2, 256, 1, A16, 256, 8, A16 * 3, None, A16 * 5, lda, A16 * 5, ldo, None)

    assert call(4) == gmi.GMI_ERR_INVALID_ARG and "leading dimension" in gmi.lib().gmi_last_error().decode()
    assert call(2) == gmi.GMI_ERR_INVALID_ARG


@pytest.mark.parametrize("ldy,ldd", [(256, 264), (512, 256)])
def test_gradient_over_the_rows(gmi, ldy, ldd):
    assert gmi.lib().gmi_moe_unpermute_bwd(4, 2, 256, 1, A16 * 2, 256, A16 * 3, None, A16 * 4, ldy, 8, A16 * 4, ldd, None, 0,
                                           None, 0, A16 * 6, None) == gmi.GMI_ERR_INVALID_ARG
    assert "leading dimension" in gmi.lib().gmi_last_error().decode()


@pytest.mark.parametrize("lda,ldda", [(512, 520), (1024, 512)])
def test_gradient_over_the_gate(gmi, lda, ldda):
    assert gmi.lib().gmi_swiglu_bwd(4, 256, 1, A16 * 2, 256, A16, lda, None, A16, ldda, None, 0, None, 0,
                                    None) == gmi.GMI_ERR_INVALID_ARG
    assert "leading dimension" in gmi.lib().gmi_last_error().decode()
