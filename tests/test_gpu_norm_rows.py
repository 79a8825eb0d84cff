"""RMS norm at rows that a workgroup takes more than one of, of lengths that
test_gpu_norm has only with few rows: the same checks with the same bounds."""
import pytest

import test_gpu_norm as norm

pytestmark = pytest.mark.gpu


# rows read twice, four units a thread, two units a thread; more rows than workgroups
@pytest.mark.parametrize("T,d,prec,res", [(4100, 16448, "bf16", "f32"), (4100, 8256, "bf16", "bf16"), (4097, 4160, "f32", "f32")])
def test_forward(T, d, prec, res):
    norm.test_forward(T, d, prec, res)


# and a wave a row, with one unit a thread and many rows, with two units and the most rows of one launch
@pytest.mark.parametrize("prec,res", norm.TYPES)
@pytest.mark.parametrize("T,d", [(600, 16448), (1100, 8256), (1025, 16384), (1030, 4160), (1030, 448), (1024, 1024), (1024, 576)])
def test_backward(T, d, prec, res):
    norm.test_backward(T, d, prec, res)


@pytest.mark.parametrize("T,d", [(600, 16448), (1100, 8256), (33000, 4160)])
def test_weight_gradient(T, d):
    norm.test_weight_gradient_of_many_rows(T, d)
