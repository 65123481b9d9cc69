"""CPU tests of the token-row operators' C ABI: pointers and sizes that it has
to refuse before any launch."""
import ctypes

import pytest

from submanifold_sparse_convolution_hash_gb300 import binding


@pytest.fixture(scope="module")
def libsc():
    from submanifold_sparse_convolution_hash_gb300 import build
    build.build()
    return binding.lib()


def test_rotation_refuses_weight_gradients_in_host_memory(libsc):
    """With no tokens as well: they are set to zero then."""
    host = (ctypes.c_float * 64)()
    p = ctypes.addressof(host)
    assert libsc.sc_qk_norm_rope_bwd(None, None, None, None, None, None, p, None, p, None, None, 0, 1, None, 0, 2, 0, 64,
                                     0, 1e-6, 1.0, 1, 0, None) == 1
    assert b"weight gradients" in libsc.sc_last_error()


def test_attention_refuses_a_scale_whose_product_with_log2_e_overflows(libsc):
    def call(scale):
        return libsc.sc_attn_fwd(None, None, None, None, None, None, None, None, 1, 4, 4, 2, 2, 64, scale, 1, 0, None)

    assert call(3e38) == 1 and b"scale" in libsc.sc_last_error()
    assert call(1.0) == 1 and b"scale" not in libsc.sc_last_error()
