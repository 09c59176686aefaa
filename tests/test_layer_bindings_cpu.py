"""The layer bindings refuse host tensors before the library sees a pointer."""
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr


class OnDevice(torch.Tensor):
    """A host tensor that says it is a CUDA tensor, for the arguments beside the one tested."""

    @property
    def is_cuda(self):
        return True


def dev(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


N, D = 2, 64


class Library:
    """In the library's place: no call may reach it with these tensors."""

    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} was called")
        return call


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(pr, "load_library", Library)


def norm_args():
    return dict(h=dev(N, D), hs=D, gate=dev(N, D), gs=D, act=0, w_post=None, res=dev(N, D), rs=D, scale=None,
                w_pre=None, s=dev(N, D), x=None, eps=1e-6, N=N, D=D)


def adjoint_args():
    a = norm_args()
    return dict(h=a["h"], hs=D, gate=a["gate"], gs=D, act=0, w_post=None, res=a["res"], rs=D, scale=None,
                w_pre=dev(D), ds=dev(N, D), dss=D, dx=dev(N, D), dxs=D, dh=dev(N, D), dg=dev(N, D), dr=None,
                dwp=None, dsc=None, dwpre=None, eps=1e-6, N=N, D=D)


@pytest.mark.parametrize("bad", ["host", "channels"])
@pytest.mark.parametrize("name", ["h", "gate", "res"])
def test_block_norm_binding_refuses(name, bad):
    a = norm_args()
    a[name] = torch.zeros(N, D) if bad == "host" else dev(N, 2 * D)[:, ::2]
    with pytest.raises(ValueError):
        pr.pararnn_block_norm(*a.values(), stream=0)


@pytest.mark.parametrize("bad", ["host", "channels"])
@pytest.mark.parametrize("name", ["h", "gate", "res", "ds", "dx"])
def test_block_norm_adjoint_bindings_refuse(name, bad):
    a, ws = adjoint_args(), dev(1 << 20, dtype=torch.uint8)
    a[name] = torch.zeros(N, D) if bad == "host" else dev(N, 2 * D)[:, ::2]
    with pytest.raises(ValueError):
        pr.pararnn_block_norm_adjoint(*a.values(), ws, stream=0)
    with pytest.raises(ValueError):
        pr.pararnn_block_norm_adjoint_ex(*a.values(), None, ws, None, stream=0)
