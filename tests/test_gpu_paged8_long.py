"""The longest segment of the 8-bit attention: a table of 2^20 pages, 2^19 chunks that one CTA
works through by itself."""
import pytest

from gpu_common import torch_cuda
from test_gpu_paged import PAGE, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages,nan", [(1 << 12, True), (1 << 20, False), (1 << 20, True)])
def test_a_pair_of_a_whole_table_in_one_segment(pages, nan):
    """One page stands for all of them, and there are as many kv heads as CTAs.  Queries are zero,
    whose weights are equal and whose sums are exact: a value of 2 in one dimension, and of 1
    at every other position in another.  Beside them 48 of 64 heads may be NaN."""
    torch = torch_cuda()
    import speculative_decoding_verify_pass_gb300 as sv
    hkv, group, hd = torch.cuda.get_device_properties(0).multi_processor_count, 64, 64
    kp = torch.zeros((1, hkv, PAGE, hd), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros((1, hkv, PAGE, hd), device="cuda")
    v[..., 3] = 2.0
    v[:, :, ::2, 40] = 1.0
    vp = v.to(torch.float8_e4m3fn)
    sc = torch.full((1, hkv, 2, PAGE), 127, dtype=torch.uint8, device="cuda")
    q = torch.zeros((1, hkv, group, hd), dtype=torch.bfloat16, device="cuda")
    if nan:
        q[:, :, 16:] = float("nan")
    tables = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    err = i32([0])
    out = sv.spec_paged_attention_fp8(q.view(1, hkv * group, hd), i32([0, 1]), i32([pages * PAGE]), tables, kp, vp, sc, 1,
                                      d_error=err).view(hkv, group, hd)
    assert err.item() == 0
    want = torch.zeros(hd, dtype=torch.bfloat16, device="cuda")
    want[3], want[40] = 2.0, 0.5
    assert torch.equal(out[:, :16], want.expand(hkv, 16, hd))
    assert torch.isnan(out[:, 16:]).all() or not nan
