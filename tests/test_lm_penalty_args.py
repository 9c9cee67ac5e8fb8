"""CPU: arguments of the logits penalties that may not be passed over."""
import pytest
import torch

import sparse_gradient_backward_amd as sgb
from sparse_gradient_backward_amd import lm

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="plans without a device")


def status(**kw):
    """What a call with these arguments ends in; SGB_ERR_HIP where it is valid
    (there is no device)."""
    p = lm.LogitsPenalty(50)
    buf = torch.zeros(128, dtype=torch.float64)
    c = dict(logits=torch.zeros(3, 50), out=torch.zeros(3, 50),
             workspace=buf[-buf.data_ptr() % 256 // 8:][:32])
    with pytest.raises(sgb.SgbError) as e:
        p.apply(**{**c, **kw})
    return e.value.name


@no_gpu
def test_no_masks_for_rows_that_have_one_each():
    masks = torch.empty(0, 2, dtype=torch.int32)
    assert status(mask=masks) == "SGB_ERR_INVALID_ARGUMENT"
    assert status(mask=torch.zeros(3, 2, dtype=torch.int32)) == "SGB_ERR_HIP"
    assert status(mask=masks, mask_index=torch.zeros(3, dtype=torch.int32)) == "SGB_ERR_HIP"


@no_gpu
def test_arguments_without_what_they_belong_to():
    """Dropped in silence, the logits would go without their biases; a mask
    index alone means nothing, as mask says whether there are masks."""
    i32 = torch.int32
    for kw in (dict(bias_values=torch.zeros(3, 2)), dict(tokens=torch.zeros(3, dtype=i32)),
               dict(bias_ids=torch.zeros(3, dtype=i32)), dict(mask=torch.zeros(2, dtype=i32)),
               dict(mask=torch.zeros(1, 2, 2, dtype=i32))):
        assert status(**kw) == "SGB_ERR_INVALID_ARGUMENT", kw
    assert status(mask_index=torch.zeros(3, dtype=i32)) == "SGB_ERR_HIP"
