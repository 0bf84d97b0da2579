"""Norm rows in numbers that leave part of a warp without a row, contiguous and as slices of wider
buffers, against the formulas in 64 bits (tolerances as in test_gpu_rmsnorm.py)."""
import pytest

pytestmark = pytest.mark.gpu

fs = pytest.importorskip("fully_sharded_gb300")
torch = pytest.importorskip("torch")

from test_gpu_rmsnorm import BF16, F32, check_backward, check_y, guarded, rand, untouched, want_forward  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")


@pytest.mark.parametrize("rows,cols,stride", [(1001, 50, 50), (1003, 33, 33), (513, 33, 33), (514, 50, 50), (1001, 41, 41),
                                              (1001, 121, 121), (1001, 50, 4097), (513, 3, 4097), (515, 100, 4097),
                                              (40001, 50, 50), (40003, 57, 63), (40001, 117, 117)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_part_of_a_warp_without_rows(rows, cols, stride, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    (_, x), (_, residual), (whole_h, h), (whole_y, y), (_, dy), (whole_dx, dx) = (
        guarded(rows, cols, dtype, stride, offset=1) for _ in range(6))
    for t in (x, residual, dy):
        t.copy_(rand(gen, rows, cols))
    gain = rand(gen, cols, dtype=F32)
    fs.fsdp_rmsnorm(x, gain, y, residual=residual, h_out=h)
    check_y(y, want_forward(x, residual, gain, 1e-6)[2], cols)
    assert torch.equal(h, (x.float() + residual.float()).to(dtype))
    assert untouched(whole_y, y) and untouched(whole_h, h)
    fs.fsdp_rmsnorm(x, gain, y)
    check_y(y, want_forward(x, None, gain, 1e-6)[2], cols)
    check_backward(dy, h, gain, residual, dx=dx)
    assert untouched(whole_dx, dx)


@pytest.mark.parametrize("cols", [768, 101, 20001])
@pytest.mark.parametrize("stride", [0, -1, -(1 << 40), 1 << 62])
def test_the_stride_of_a_single_row_does_not_matter(cols, stride):
    import ctypes

    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, dy, dh, gain = (rand(gen, *s) for s in ((1, cols), (1, cols), (1, cols), (cols,)))
    y, h, dx, rstd, dgain = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty(1, device="cuda"), torch.empty_like(gain)
    stream = torch.cuda.current_stream().cuda_stream
    a = fs.RmsNormArgs(1, cols, stride, stride, stride, stride, 0, 0, 0, 0, 1e-6)
    assert fs._lib.fsdp_rmsnorm(ctypes.byref(a), x.data_ptr(), dh.data_ptr(), gain.data_ptr(), h.data_ptr(), y.data_ptr(), None,
                                rstd.data_ptr(), stream) == fs.FSDP_OK
    check_y(y, want_forward(x, dh, gain, 1e-6)[2], cols)
    b = fs.RmsNormBackwardArgs(1, cols, stride, stride, stride, stride, 0, 0)
    workspace = torch.empty(fs.fsdp_rmsnorm_backward_workspace(1, cols), dtype=torch.uint8, device="cuda")
    assert fs._lib.fsdp_rmsnorm_backward(ctypes.byref(b), dy.data_ptr(), h.data_ptr(), gain.data_ptr(), rstd.data_ptr(), dh.data_ptr(),
                                         dx.data_ptr(), dgain.data_ptr(), workspace.data_ptr(), workspace.numel(), stream) == fs.FSDP_OK
    plain, plain_gain = torch.empty_like(dx), torch.empty_like(gain)
    fs.fsdp_rmsnorm_backward(dy, h, gain, rstd, plain, plain_gain, workspace, dh=dh)
    assert torch.equal(dx, plain) and torch.equal(dgain, plain_gain)
    out, again = torch.empty(1, cols, dtype=BF16, device="cuda"), torch.empty(1, cols, dtype=BF16, device="cuda")
    batch = fs.NewtonSchulzBatch([x], [out])
    batch.array[0].source_stride = batch.array[0].out_stride = stride
    room = torch.empty(fs.fsdp_newton_schulz_workspace(batch), dtype=torch.uint8, device="cuda")
    fs.fsdp_newton_schulz(batch, room)
    fs.fsdp_newton_schulz(fs.NewtonSchulzBatch([x], [again]), room)
    assert torch.equal(out, again)
