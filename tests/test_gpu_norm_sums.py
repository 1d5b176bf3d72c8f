"""The norm's column sums between workgroups, on the GPU: fp64."""
import pytest
import torch

from gpu_util import load_binding, needs_gpu

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.fixture(scope="module")
def B():
    return load_binding()


# H, dtype, rows of a workgroup, workgroups to a compute unit: rows of 16 and 64
# threads, of a workgroup, and wide rows
@pytest.mark.parametrize("H,dtype,rows,groups", [
    (8, torch.float32, 32, 1), (1024, torch.float32, 8, 1), (2048, torch.bfloat16, 8, 1),
    (4096, torch.float32, 1, 2), (4104, torch.bfloat16, 1, 2), (8192, torch.float32, 1, 2), (8200, torch.bfloat16, 1, 2)])
def test_norm_joins_the_workgroups_sums_in_64_bits(B, H, dtype, rows, groups):
    """One pass of every workgroup: 2^40 in one of them, -2^40 in another, ones in all
    others' rows.  Each workgroup's sum is exact in fp32 (one value, or at most 32
    ones), and so is the result in fp64, in any order; an fp32 sum that holds 2^40
    has steps of 2^17 and drops every one that is added to it there."""
    blocks = groups * torch.cuda.get_device_properties(0).multi_processor_count
    print(f"[gpu-test] norm sums {H} {dtype} {blocks}", flush=True)
    T, other = rows * blocks, rows * (blocks * 5 // 8)
    dy = torch.ones(T, H, dtype=dtype, device="cuda")
    for at, value in ((0, 2.0 ** 40), (other, -2.0 ** 40)):
        dy[at:at + rows] = 0
        dy[at] = value
    want = float(torch.tensor(float(T - 2 * rows)).to(dtype))
    s, rstd = torch.ones(T, H, dtype=dtype, device="cuda"), torch.ones(T, device="cuda")
    ws = B.new_workspace(B.moe_norm_backward_workspace_size(T, H, dtype), "cuda")
    ws.fill_(0xFF)
    dw, db = torch.empty(H, dtype=dtype, device="cuda"), torch.empty(H, dtype=dtype, device="cuda")
    B.moe_norm_backward(dy, s, None, rstd, ws, kind="rms", dweight=dw, dbias=db)
    assert (dw == want).all() and (db == want).all()
