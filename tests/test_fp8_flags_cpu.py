"""The FP8 forwards' test flag in x_dt, without a GPU."""
import pytest

import sparse_quantized_rank_b200 as C

P = 1 << 20                                   # a 256-byte aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    from sparse_quantized_rank_b200 import build
    build.build()
    return C.lib()


def test_flag_changes_no_check(lib):
    """With the flag a call is checked as without it: a known type is taken (here
    with no tokens, so that nothing is launched), any other refused."""
    def call(x_dt, ldx=300, tokens=0, grouped=False):
        head, mid = (200, 300) + ((3,) if grouped else ()), (P,) if grouped else ()
        f = lib.cql_fp8_grouped_forward if grouped else lib.cql_fp8_linear_forward
        return f(*head, P, P, x_dt, ldx, *mid, P, C.CQL_DT_F32, 200, tokens, P, 1 << 20, P, None)
    flag = C.CQL_FLAG_DEBUG_SKIP_X
    for grouped in (False, True):
        for dt in (C.CQL_DT_F32, C.CQL_DT_F16, C.CQL_DT_BF16):
            assert call(dt | flag, grouped=grouped) == C.CQL_OK
            assert call(dt | flag, ldx=299, grouped=grouped) == C.CQL_ERR_ARG
        assert call(C.CQL_DT_FP8_BLOCK | flag, 0, grouped=grouped) == C.CQL_OK
        assert call(C.CQL_DT_FP8_BLOCK | flag, 300, grouped=grouped) == C.CQL_ERR_ARG
        for dt in (4 | flag, 2 * flag, 0x200 | flag, -1):
            assert call(dt, grouped=grouped) == C.CQL_ERR_ARG, hex(dt)
