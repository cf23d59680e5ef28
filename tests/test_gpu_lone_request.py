"""Decode of a batch with one non-empty request: its blocks are the whole
stream of a q-head group, so a warp's range runs from the last blocks of one
group into the first blocks of the same request for the next group."""
import numpy as np
import pytest

import oracle
import synthetic

pytestmark = pytest.mark.gpu

from gpu_harness import assert_close, fill_pool, out_to_f64, run_step  # noqa: E402


@pytest.mark.parametrize("kv_dtype", ["f16", "bf16", "int8", "int4"])
@pytest.mark.parametrize("lens", [[641], [0, 1043, 0], [17], [530]])
def test_one_request(gpu, kv_dtype, lens):
    """41 blocks of a request in ranges of 4: every tenth range straddles two groups."""
    wl = synthetic.custom(f"lone_{kv_dtype}", kv_dtype, lens, 16, 8, seed=91)
    pool = fill_pool(wl)
    out, _, dev_err = run_step(wl, pool)
    assert gpu.kvq_check_error(dev_err) == 0
    _, oout = oracle.run_workload(wl)
    assert_close(out_to_f64(out), np.asarray(oout))
