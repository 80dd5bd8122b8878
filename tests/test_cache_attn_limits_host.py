"""The largest numbers of rows that attention over a paged cache takes, without a GPU: the kernels count rows in
32 bits, rounded up to tiles of 128 and to whole tokens."""
import pytest

from test_cache_host import ashape, attend, cshape, ref


@pytest.fixture(scope="module")
def tp():
    from tensor_transformer_mlp_tma_gb300 import build
    build.build()
    from tensor_transformer_mlp_tma_gb300 import tpmlp
    return tpmlp


def test_rows_near_the_end_of_32_bits(tp):
    for heads in (1, 2, 8, 33, 65536):
        most = ((1 << 31) - 1025) // heads - 1
        for T, good in ((most, True), (most + 1, False)):
            s, c = ashape(tp, T=T, heads=heads), cshape(tp, kv=1)
            assert (tp.lib.tpmlp_cache_attn_workspace_bytes(ref(s), ref(c)) > 0) == good, (T, heads)
            if not good:
                assert attend(tp, s, c) == tp.ERR_INVALID_ARG
        # rows to the end of a tile, and from there to the end of a token
        assert most * heads + 127 + heads - 1 < 1 << 31
