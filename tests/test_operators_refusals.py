"""Further refusals of the linear-attention and query/key-norm entry points, on the CPU: all are found on the host before
anything is launched."""
import pytest

import bit_recurrent_state_pace_b200 as pace


def test_debug_limits_of_the_chunk_kernel():
    for tries, extra in ((99, 0), (200001, 0), (100, 8), (100, 32), (1001, 16), (0, 16)):
        with pytest.raises(pace.PaceError) as e:
            pace.pace_debug_linattn_wait(tries, extra)
        assert e.value.status == pace.PACE_ERR_INVALID_ARG
    pace.pace_debug_linattn_wait(100, 0)
    pace.pace_debug_linattn_wait(0, 0)
