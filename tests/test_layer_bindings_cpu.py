"""The layer bindings refuse host tensors, and tensors of another device than the
current one, before the library sees a pointer."""
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on the first CUDA device, for the arguments beside the one tested."""
    index = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)


class Elsewhere(OnDevice):
    index = 1


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
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


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


B, T, G = 2, 4, 2


def solve_args():
    return dict(u=dev(B, T, G, D), lam=None, bias=dev(G, D), h0=dev(B, D), reset=dev(B, T, dtype=torch.uint8),
                h=dev(B, T, D))


def gradient_args():
    return dict(solve_args(), dLdh=dev(B, T, D), du=dev(B, T, G, D), dlam=None, dbias=dev(G, D), dh0=dev(B, D))


def step_args():
    return dict(u=dev(B, G, D), lam=None, bias=dev(G, D), h_prev=dev(B, D), h_next=dev(B, D))


def _calls():
    ws = lambda: dev(1 << 20, dtype=torch.uint8)  # noqa: E731
    word = lambda: dev(1, dtype=torch.int32)  # noqa: E731
    return {
        "linrec_solve": lambda: solve_args(),
        "linrec_solve_ex": lambda: dict(solve_args(), status=word(), opts=None),
        "linrec_adjoint": lambda: dict(gradient_args(), ws=ws()),
        "linrec_adjoint_ex": lambda: dict(gradient_args(), status=word(), ws=ws(), opts=None),
        "linrec_step": lambda: step_args(),
        "block_norm": lambda: norm_args(),
        "block_norm_adjoint": lambda: dict(adjoint_args(), ws=ws()),
        "block_norm_adjoint_ex": lambda: dict(adjoint_args(), status=word(), ws=ws(), opts=None),
    }


CASES = [(c, k) for c, a in _calls().items() for k, v in a().items() if torch.is_tensor(v)]


def call(name, args):
    cell = () if name.startswith("block") else (pr.PARARNN_LIN_GRU,)
    return getattr(pr, "pararnn_" + name)(*cell, *args.values(), stream=0)


@pytest.mark.parametrize("name,arg", CASES)
def test_bindings_refuse_another_device(name, arg):
    args = _calls()[name]()
    args[arg] = args[arg].as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        call(name, args)


@pytest.mark.parametrize("name", _calls())
def test_bindings_reach_the_library_otherwise(name):
    with pytest.raises(AssertionError, match="pararnn_" + name):
        call(name, _calls()[name]())
