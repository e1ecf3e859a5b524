"""Which kernel a call of the embedding, layer norm and the matrices' updates reaches, by
the name that ``last_kernel`` gives, beside each limit of the choice."""
import pytest
import torch

import sharded_optimizer_step_gb300 as ss

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ss.build()
    yield
    assert ss.device_status() == 0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(rows, cols, dtype, stride=None, shift=0):
    stride = stride or cols
    buf = torch.zeros(rows * stride + shift + 16, dtype=dtype, device=DEV)
    return buf[shift:shift + rows * stride].view(rows, stride)[:, :cols].normal_(generator=_gen(1))


@pytest.mark.parametrize("dtype,cols,stride,shift,out_stride,forward,backward", [
    (BF, 768, 768, 0, 768, "layer_norm_vectors", "layer_norm_staged_grad"),
    (BF, 770, 776, 0, 776, "layer_norm_vectors", "layer_norm_staged_grad"),
    (BF, 770, 776, 0, 770, "layer_norm_vectors, turned", "layer_norm_staged_grad, by elements"),
    (F32, 5003, 5004, 0, 5003, "layer_norm_vectors, turned",
     "layer_norm_staged_grad, by elements"),
    (BF, 8192, 8192, 0, 8192, "layer_norm_vectors", "layer_norm_staged_grad"),
    (BF, 8200, 8200, 0, 8200, "layer_norm_vectors", "layer_norm_wide_grad"),
    (BF, 16384, 16384, 0, 16384, "layer_norm_vectors", "layer_norm_wide_grad"),
    (BF, 16392, 16392, 0, 16392, "layer_norm_wide", "layer_norm_wide_grad"),
    (BF, 769, 769, 0, 769, "layer_norm_elements", "layer_norm_elements_grad"),
    (BF, 768, 768, 1, 768, "layer_norm_elements", "layer_norm_elements_grad"),
    (BF, 4096, 4097, 0, 4096, "layer_norm_elements", "layer_norm_elements_grad"),
    (BF, 4097, 4097, 0, 4097, "layer_norm_elements", "layer_norm_wide_grad"),
    (BF, 8193, 8193, 0, 8193, "layer_norm_wide", "layer_norm_wide_grad"),
])
def test_layer_norm_names(dtype, cols, stride, shift, out_stride, forward, backward):
    name = " <bf16>" if dtype is BF else " <f32>"
    x = _rows(5, cols, dtype, stride, shift)
    w = torch.randn(cols, device=DEV, generator=_gen(2))
    y = ss.layer_norm(x, w, out=_rows(5, cols, dtype, out_stride))
    assert ss.last_kernel() == forward + name
    d = ss.layer_norm_grad(x, x, y.mean, y.rstd, w, d_x=_rows(5, cols, dtype, out_stride),
                           d_weight=torch.empty_like(w))
    assert ss.last_kernel() == backward + name
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    want = torch.nn.functional.layer_norm(xd, (cols,), wd)
    want.backward(x.double())
    # a few steps of the type beside fp32's sums: a wrong path is off by whole elements
    tol = 4 * torch.finfo(dtype).eps
    for got, ref in ((y.out, want.detach()), (d.d_x, xd.grad), (d.d_weight, wd.grad)):
        assert float((got.double() - ref).abs().max()) <= tol * float(ref.abs().max())


def test_layer_norm_names_without_rows_or_d_x():
    x, w = _rows(5, 9000, BF), torch.randn(9000, device=DEV)
    y = ss.layer_norm(x, w)
    ss.layer_norm_grad(x, x, y.mean, y.rstd, w, d_weight=torch.empty_like(w))
    assert ss.last_kernel() == "layer_norm_wide_columns <bf16>"
    ss.layer_norm_grad(x[:0], x[:0], y.mean[:0], y.rstd[:0], w, d_weight=torch.empty_like(w))
    assert ss.last_kernel() == "layer_norm_columns <bf16>"


def test_embedding_names():
    ids = torch.tensor([1, 3, 1], device=DEV)
    for dim, how in ((16, "vectors"), (17, "elements")):
        table = _rows(5, dim, BF)
        out = ss.embedding(table, ids)
        assert ss.last_kernel() == f"embedding_lookup<bf16> ({how})"
        ss.embedding_grad(out, ids, torch.empty(5, dim, device=DEV))
        assert ss.last_kernel() == f"embedding_sum<bf16, f32> ({how})"


def test_matrices_names():
    us = [torch.randn(40, 30, device=DEV), torch.randn(3, 700, device=DEV)]
    ss.orthogonalize(us)
    assert ss.last_kernel() == "matrix_rounds<128, 64>"
    ss.layer_norm(us[1])
    opt = ss.TensorMuon([u.to(BF) for u in us], ss.Muon())
    opt.step(us)
    assert ss.last_kernel() == "matrix_rounds<128, 64>"
    ss.layer_norm(us[1])
    ss.orthogonalize([u[:0] for u in us])                  # nothing is launched
    assert ss.last_kernel() == "layer_norm_vectors <f32>"
