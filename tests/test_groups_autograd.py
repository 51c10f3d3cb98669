"""The autograd functions behind the grouped products: what they save, pass on and refuse.

The library's calls are replaced by their formulas on the CPU, in 64 bits; test_gpu_groups_autograd.py has
the calls themselves.
"""
import pytest
import torch

import tiled_dense_gemm_relu_amd as gr
from tiled_dense_gemm_relu_amd import groups

ENDS = [2, 2, 5]                    # three groups, one of them empty, and a row of none


@pytest.fixture
def formulas(monkeypatch):
    def spans(ends):
        return list(zip([0, *ends.tolist()], ends.tolist()))

    def forward(a, b, ends, b_layout=gr.B_KN, relu=True, config=-1, workspace=None):
        assert not torch.is_grad_enabled()
        y = a.new_zeros((a.shape[0], b.shape[1 if b_layout == gr.B_NK else 2]))
        for g, (lo, hi) in enumerate(spans(ends)):
            y[lo:hi] = a[lo:hi] @ (b[g].t() if b_layout == gr.B_NK else b[g])
        return y.clamp_min(0) if relu else y

    def backward(dc, c, a, b, ends, b_layout=gr.B_KN, relu=True, need_da=True, need_db=True):
        assert dc.is_contiguous() and (c is None) == (not relu) and (a is None) == (not need_db)
        assert (b is None) == (not need_da)
        d = dc * (c > 0) if relu else dc
        da = db = None
        if need_da:
            da = dc.new_zeros((dc.shape[0], b.shape[2 if b_layout == gr.B_NK else 1]))
        if need_db:
            db = dc.new_zeros((len(ends), dc.shape[1], a.shape[1]) if b_layout == gr.B_NK
                              else (len(ends), a.shape[1], dc.shape[1]))
        for g, (lo, hi) in enumerate(spans(ends)):
            if need_da:
                da[lo:hi] = d[lo:hi] @ (b[g] if b_layout == gr.B_NK else b[g].t())
            if need_db:
                db[g] = d[lo:hi].t() @ a[lo:hi] if b_layout == gr.B_NK else a[lo:hi].t() @ d[lo:hi]
        return da, db
    monkeypatch.setattr(groups, "gemm_relu_grouped", forward)
    monkeypatch.setattr(groups, "gemm_relu_grouped_backward", backward)
    return groups._functions()[0].apply


@pytest.mark.parametrize("relu", [True, False])
@pytest.mark.parametrize("layout", [gr.B_KN, gr.B_NK])
@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
def test_gradients_against_differences(formulas, needs, layout, relu):
    g = torch.Generator().manual_seed(1)
    a = torch.randn((6, 4), generator=g, dtype=torch.float64).requires_grad_(needs[0])
    b = torch.randn((3, 3, 4) if layout == gr.B_NK else (3, 4, 3), generator=g, dtype=torch.float64).requires_grad_(needs[1])
    ends = torch.tensor(ENDS, dtype=torch.int32)

    def call(a, b):
        return formulas(a, b, ends, layout, relu, -1, None)
    # (no sum is within 1e-3 of ReLU's edge with these numbers, and differences step by 1e-6)
    assert torch.autograd.gradcheck(call, (a, b))
    call(a, b).sum().backward()                         # an expanded gradient reaches the call whole
    assert (a.grad is not None) == needs[0] and (b.grad is not None) == needs[1]


def test_second_derivatives_are_refused(formulas):
    a = torch.ones((5, 2), dtype=torch.float64, requires_grad=True)
    b = torch.ones((3, 2, 2), dtype=torch.float64, requires_grad=True)
    y = formulas(a, b, torch.tensor(ENDS, dtype=torch.int32), gr.B_KN, True, -1, None)
    grad, = torch.autograd.grad((y * y).sum(), a, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.sum().backward()


def test_adapters_have_no_gradient(monkeypatch):
    monkeypatch.setattr(groups, "gemm_relu_adapters", lambda x, w, *rest, **kw: x @ w)
    x, w = torch.ones((2, 3)), torch.ones((3, 4), requires_grad=True)
    y = groups._functions()[1].apply(x, w, *[None] * 9)
    assert y.requires_grad
    with pytest.raises(NotImplementedError, match="no_grad"):
        y.sum().backward()


def test_out_is_refused_where_a_gradient_is_asked_for():
    with pytest.raises(RuntimeError, match="no_grad"):
        groups._differentiable(groups._functions()[0], 0, torch.ones(1), None)
