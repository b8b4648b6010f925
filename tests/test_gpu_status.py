"""The error word's reports do not hide one another: a wait that gave up (a TMA stage withheld by the
test hook) and a slot out of range, recorded by two calls before one sq_sync_status()."""
import pytest
import torch

from w8a8_quantized_gemm_b200 import sq

from _gpu import empty

pytestmark = pytest.mark.gpu


def _withheld_stage():
    M, N, K = 256, 512, 1024
    a, w = torch.ones(M, K, dtype=torch.int8, device="cuda"), torch.ones(N, K, dtype=torch.int8, device="cuda")
    ws = sq.workspace(sq.SQ_OP_INT8_GEMM_DEQUANT, M, N, K)
    sq.sq_debug_arm_fault(1, 50_000_000)  # 50 ms per wait
    sq.sq_int8_gemm_dequant(a, w, torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), sq.SQ_PER_CHANNEL, None,
                            empty((M, N), torch.bfloat16), None, ws)


def _bad_slot():
    k = torch.zeros(2, 1, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    sq.sq_rope_kv_append(None, x, x, None, None, None, torch.tensor([8], dtype=torch.int32, device="cuda"),
                         sq.KvCache(k[0], k[1]), None)


@pytest.mark.parametrize("calls", [(_withheld_stage, _bad_slot), (_bad_slot, _withheld_stage)])
def test_a_timeout_is_not_hidden_by_an_index(calls):
    sq.sq_sync_status()  # clean slate
    for call in calls:
        call()
    for status in (sq.SQ_ERR_TIMEOUT, sq.SQ_ERR_BOUNDS):
        with pytest.raises(sq.SqError) as ei:
            sq.sq_sync_status()
        assert ei.value.status == status
    sq.sq_sync_status()  # both are cleared
