"""Edges of the decoder operators on the GPU, against the float64 definition:
partial results of the two paged kernels side by side, rows that see few keys,
sink gradients of many sequences, streams."""
import pytest
import torch

from sparse_attention_banded_b200 import build, lf
from tests._window_ref import check, half_step, reference, subnormal_half_step
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lf.lib()
    lf.lf_device_status(reset=True)
    yield


@pytest.fixture(autouse=True)
def _status():
    yield
    assert lf.lf_device_status(reset=True) == 0


@pytest.mark.parametrize("q,kv,Hq,Hkv", [
    ([1, 150, 1, 3, 0, 1, 40, 2], [5000, 3000, 30, 7000, 9, 1, 2500, 4097], 8, 2),    # slots by sequence
    ([1, 17, 1], [6000, 5000, 100], 2, 2),                                            # slots by sequence, 16 each
    ([16, 17, 16, 15, 1], [3000, 2000, 40, 2500, 4000], 3, 3),                        # slots by token
    ([5, 6, 5, 1], [3000, 5000, 7, 2500], 3, 1)])                                     # the same, three heads a group
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_pieces_of_both_kernels_in_one_call(dtype, q, kv, Hq, Hkv):
    """Contexts cut by the decode kernel next to ones cut by the tensor-core
    kernel, in a table wide enough for several pieces of each."""
    c = Case(q, kv, Hq, Hkv, 16, dtype, seed=len(q) + Hq, extra=1000)
    n, T, wide = len(q), c.q.shape[0], c.table.shape[1]
    short = lf.lf_paged_attention_workspace_bytes(n, Hq, Hkv, T, 16 // (Hq // Hkv), wide, 16, c.w, 0)
    both = lf.lf_paged_attention_workspace_bytes(n, Hq, Hkv, T, max(q), wide, 16, c.w, 0)
    assert 0 < short < both
    c.run().check()
