"""GPU: logits penalties at the ends: every bit pattern of an untouched logit,
a set of no masks."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from sparse_gradient_backward_amd import lm as m
    return m


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_untouched_logits_keep_their_bits(lm, dt):
    """All 65536 patterns; a NaN stays a NaN."""
    V = 65536
    bits = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(dt).reshape(1, V)
    p = lm.LogitsPenalty(V)
    out = torch.empty_like(x)
    p.apply(x, out, workspace=p.workspace(1))
    nan = x.isnan()
    assert torch.equal(out.isnan(), nan)
    assert torch.equal(out.view(torch.int16)[~nan], x.view(torch.int16)[~nan])
    quiet = nan & ((x.view(torch.int16) & (0x40 if dt is torch.bfloat16 else 0x200)) != 0)
    assert torch.equal(out.view(torch.int16)[quiet], x.view(torch.int16)[quiet])


def test_fp32_logits_keep_their_bits(lm):
    V = 70001
    g = torch.Generator(device="cuda").manual_seed(1)
    bits = torch.randint(-2**31, 2**31, (3, V), generator=g, device="cuda").int()
    bits[1] = torch.arange(V, device="cuda").int()              # the smallest subnormals
    bits[2] = torch.arange(V, device="cuda").int() + 0x7f7fff00  # infinity, signalling and quiet NaNs
    x = bits.view(torch.float32)
    p = lm.LogitsPenalty(V)
    out = torch.empty_like(x)
    p.apply(x, out, workspace=p.workspace(3))
    assert torch.equal(out.view(torch.int32), bits)


def test_an_index_into_no_masks_is_reported(lm):
    V = 100
    x = torch.randn(3, V, device="cuda")
    p = lm.LogitsPenalty(V)
    ws, out = p.workspace(3), torch.empty_like(x)
    masks = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    for index, status in (([-1, -1, -1], "SGB_OK"), ([-1, 0, -1], "SGB_ERR_INDEX_OUT_OF_RANGE")):
        i = torch.tensor(index, dtype=torch.int32, device="cuda")
        p.apply(x, out, mask=masks, mask_index=i, workspace=ws)
        assert p.device_status(ws) == status
        assert torch.equal(out, x)
