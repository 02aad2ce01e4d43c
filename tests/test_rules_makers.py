"""The binding's makers of rules at the ends of binary32."""
import numpy as np
import pytest

import token_sampling_amd as sv


# The largest binary32 value is 2^128 - 2^104 and its step 2^104: doubles from half a
# step above it on round to infinity, those below to it.
@pytest.mark.parametrize("value", [1e300, 3.5e38, 2.0**128 - 2.0**103, float("inf"), float("nan")])
def test_bias_out_of_binary32(value):
    """A bias that becomes +inf when it is narrowed would fail its session."""
    with pytest.raises(ValueError):
        sv.make_bias([{0: 1.0}, {2: value}], 4, device="cpu")


def test_bias_values():
    big = float(np.finfo(np.float32).max)
    b = sv.make_bias([{3: 2.0**128 - 2.0**103 * 1.001, 0: -big}, None, {1: -1e300, 2: 0.1}], 4, device="cpu")
    assert b.offsets.tolist() == [0, 2, 2, 4] and b.ids.tolist() == [0, 3, 1, 2]
    assert b.values.tolist() == [-big, big, float("-inf"), float(np.float32(0.1))]
    none = sv.make_bias([None, {}], 4, device="cpu")
    assert none.offsets.tolist() == [0, 0, 0] and none.values.shape == (0,) and none.ids.shape == (0,)
