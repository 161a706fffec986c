"""GPU: MX-FP4 quantisation, byte for byte against the definition, the oracle's encoder's rule
and the dispatch's own encoding."""
import numpy as np
import pytest
import torch

import more_reference as ref
from gpu_helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import combine_topk_ids_amd.moe as m
    return m


def run(moe, x):
    rows, cols = x.shape
    codes = torch.full((rows, cols // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, codes, scales)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (7, 544), (333, 64), (64, 4096), (5, 8192 + 32), (1000, 160)])
def test_against_the_definition(moe, rows, cols):
    say(f"[quantize] {rows} x {cols}")
    g = torch.Generator("cuda").manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-130, 120, (rows, 1), generator=g, device="cuda").float())
    x[torch.rand(rows, cols, generator=g, device="cuda") < 0.05] = 0
    x = x.bfloat16()
    codes, scales = run(moe, x)
    want = ref.mx_encode(x.float().cpu().numpy())
    assert np.array_equal(scales, want[1]) and np.array_equal(codes, want[0])


def test_every_bf16_value(moe):
    """All 65,536 patterns, in blocks under every exponent of the block's maximum."""
    bits = np.arange(65536, dtype=np.uint16)
    for top in (0x0001, 0x0080, 0x3F80, 0x40E0, 0x7F7F):
        mag = bits & 0x7FFF
        # values above the block's maximum (and infinities, NaNs) are left out
        keep = bits[mag <= top]
        keep = np.concatenate([keep, np.zeros(-len(keep) % 31, dtype=np.uint16)]).reshape(-1, 31)
        rows = np.concatenate([keep, np.full((len(keep), 1), top, dtype=np.uint16)], axis=1)
        x = torch.from_numpy(rows.view(np.int16)).cuda().view(torch.bfloat16)
        codes, scales = run(moe, x)
        want = ref.mx_encode((rows.astype(np.uint32) << 16).view(np.float32))
        assert np.array_equal(scales, want[1]) and np.array_equal(codes, want[0]), hex(top)


def test_blocks_with_nan_and_infinity(moe):
    x = torch.randn(40, 96, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    clean = run(moe, x)
    x[3, 40] = float("nan")
    x[9, 0] = float("inf")
    x[11, 95] = -float("inf")
    codes, scales = run(moe, x)
    for r in range(40):
        for b in range(3):
            bad = (r, b) in ((3, 1), (9, 0), (11, 2))
            block = codes[r, 16 * b:16 * b + 16]
            assert (scales[r, b] == 255) == bad
            assert not block.any() if bad else np.array_equal(block, clean[0][r, 16 * b:16 * b + 16])


def test_the_dispatchs_encoding(moe):
    """What moe_dispatch writes for a token is what this call makes of its row."""
    n, h = 50, 416
    x = torch.randn(n, h, generator=torch.Generator("cuda").manual_seed(7), device="cuda").bfloat16()
    p = moe.problem(n, h, 1, 1, 1, fmt="mxfp4")
    plan = moe.alloc_plan(p)
    payload, scales = moe.alloc_payload(p)
    moe.moe_plan_and_dispatch(p, torch.zeros(n, 1, dtype=torch.int32, device="cuda"), plan, x, payload, scales)
    torch.cuda.synchronize()
    codes, sc = run(moe, x)
    assert np.array_equal(payload.cpu().numpy(), codes) and np.array_equal(scales.cpu().numpy(), sc)


def test_past_32_bit_offsets(moe):
    """An array of more than 2^32 bytes: its last rows are the rows alone."""
    cols, rows = 8192, (1 << 31) // 8192 + 67
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator("cuda").manual_seed(3))
    codes = torch.full((rows, cols // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mxfp4(x, codes, scales)
    for part in (slice(0, 64), slice(rows // 2, rows // 2 + 64), slice(rows - 64, rows)):
        c, s = run(moe, x[part].contiguous())
        assert np.array_equal(codes[part].cpu().numpy(), c) and np.array_equal(scales[part].cpu().numpy(), s)


def test_no_rows(moe):
    moe.moe_quantize_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"),
                           torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda"))


def test_binding_refusals(moe):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    c, s = torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        moe.moe_quantize_mxfp4(x.t(), c, s)
    with pytest.raises(ValueError, match="elements"):
        moe.moe_quantize_mxfp4(x, c[:3], s)
    with pytest.raises(ValueError, match="elements"):
        moe.moe_quantize_mxfp4(x, c, s[:3])
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_quantize_mxfp4(x.float(), c, s)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_mxfp4(x[:, :48].contiguous(), c, s)
