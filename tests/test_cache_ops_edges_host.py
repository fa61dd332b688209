"""What mfa_cache_compact refuses where K and V lie in one buffer, on the host: no call here gets past
its checks, so none touches a GPU."""
import pytest

from mask_aware_block_mfa_b200 import binding as B

from .test_cache_ops_host import PTR, compact_call, lib, tensor  # noqa: F401  (lib: a fixture)

SHAPE = (2, 3, 50, 64)  # contiguous: 9600, 3200, 64, 1
OUT = 1 << 32


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("shift", [64, -64, 128, 49 * 64, 3200, 2 * 3200, 9600, -9600, 9600 + 3200 + 64, 9600 + 2 * 3200 + 49 * 64,
                                   64 + 8, 3200 - 8, 9600 * 2 - 8])
def test_rows_of_v_that_are_rows_of_k_are_refused(lib, in_place, shift):  # noqa: F811
    """V is K moved by whole rows, heads or batches (and by less than a row more)."""
    a, b = tensor(SHAPE, OUT), tensor(SHAPE, OUT + 2 * shift)
    if in_place:
        assert compact_call(lib, k=a, v=b, ko=a, vo=b) == B.MFA_ERR_INVALID_ARG
    else:
        assert compact_call(lib, k=tensor(SHAPE), v=tensor(SHAPE, PTR * 2), ko=a, vo=b) == B.MFA_ERR_INVALID_ARG


@pytest.mark.parametrize("shift,strides", [
    (50 * 64, (3 * 2 * 50 * 64, 50 * 64, 64, 1)),       # V's heads begin where K's second one does
    (3 * 64, (50 * 2 * 3 * 64, 64, 3 * 64, 1)),         # token by token: V is K one token on
    (5 * 64 + 8, (50 * 2 * 3 * 64, 64, 2 * 3 * 64, 1)),  # K and V of a token side by side, V a few columns into the next token's K
])
def test_interleaved_tensors_that_meet_are_refused(lib, shift, strides):  # noqa: F811
    a, b = tensor(SHAPE, OUT, stride=strides), tensor(SHAPE, OUT + 2 * shift, stride=strides)
    assert compact_call(lib, k=a, v=b, ko=a, vo=b) == B.MFA_ERR_INVALID_ARG
    assert compact_call(lib, k=tensor(SHAPE), v=tensor(SHAPE, PTR * 2), ko=a, vo=b) == B.MFA_ERR_INVALID_ARG


def test_tensors_of_unlike_strides_that_meet_are_refused(lib):  # noqa: F811
    """Head by head and token by token over the same elements."""
    a, b = tensor(SHAPE, OUT), tensor(SHAPE, OUT, stride=(9600, 64, 3 * 64, 1))
    assert compact_call(lib, k=a, v=b, ko=a, vo=b) == B.MFA_ERR_INVALID_ARG
    b = tensor(SHAPE, OUT + 2 * (9600 - 64), stride=(9600, 64, 3 * 64, 1))
    assert compact_call(lib, k=tensor(SHAPE), v=tensor(SHAPE, PTR * 2), ko=a, vo=b) == B.MFA_ERR_INVALID_ARG
