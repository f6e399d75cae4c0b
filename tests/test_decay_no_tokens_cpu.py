"""Packed decay calls without tokens still launch kernels that read log_decay, so a missing one
is refused before any launch (CPU only)."""
import pytest

import chunked_gated_delta_07_gb300 as gdr
from chunked_gated_delta_07_gb300 import _build
from test_operator_refusals import bwd, fwd


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("dtype", [gdr.GDR_BF16, gdr.GDR_F32])
def test_packed_call_without_tokens_needs_the_decays(call, dtype):
    assert call(T=0, log_decay=None, cu_seqlens=10 << 20, dtype=dtype) == gdr.GDR_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [fwd, bwd])
def test_dense_call_without_tokens_does_not(call):
    # nothing to pass on either: the call returns before it needs a device
    assert call(T=0, log_decay=None) == gdr.GDR_OK


@pytest.mark.parametrize("call", [fwd, bwd])
def test_tensor_core_path_takes_no_tokens(call):
    """As the other calls' does: there is nothing that it could not run."""
    assert call(T=0, path=gdr.GDR_PATH_TC) == gdr.GDR_OK
    assert call(T=0, path=gdr.GDR_PATH_TC, dtype=gdr.GDR_F32) == gdr.GDR_ERR_UNSUPPORTED
