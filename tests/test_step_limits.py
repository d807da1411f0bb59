"""Sizes past the documented limits of the training step's operators, on the CPU: the
workspace queries say UNSUPPORTED as the calls do."""
import pytest

nf4 = pytest.importorskip("bit_quantized_fine_nf4_amd")

INV, UNS = nf4.QLORA_ERR_INVALID_VALUE, nf4.QLORA_ERR_UNSUPPORTED
NORM, LOSS = (nf4.QLORA_OP_NORM_BWD,), (nf4.QLORA_OP_LOSS_FWD, nf4.QLORA_OP_LOSS_BWD)


@pytest.mark.parametrize("ops,sizes,status", [
    (NORM, (4, 16385), UNS), (NORM, (1 << 40, 64), UNS), (NORM, (0, 64), INV), (NORM, (4, 0), INV),
    (LOSS, (4, (1 << 20) + 64, 10), UNS), (LOSS, (4, 64, (1 << 24) + 1), UNS), (LOSS, ((1 << 24) + 1, 64, 10), UNS),
    (LOSS, (1 << 20, 64, 1 << 20), UNS), (LOSS, (0, 64, 10), INV), (LOSS, (4, 65, 10), INV), (LOSS, (4, 64, 0), INV),
])
def test_workspace_queries(ops, sizes, status):
    for op in ops:
        with pytest.raises(nf4.QloraError) as e:
            nf4.workspace_size(op, *sizes)
        assert e.value.status == status
