"""The forms in which grad_norm, grad_scale and grad_clip take gradients, with a workspace and without (no GPU: the library only
records what it is handed)."""
import pytest
import torch

from tests.test_layer_binding import F32, U8, _grad, _z, recorded  # noqa: F401  (a fixture)


def _calls(layer, workspace):
    return {"mxfp4_grad_norm": lambda grads: layer.grad_norm(grads, workspace=workspace),
            "mxfp4_grad_clip": lambda grads: layer.grad_clip(grads, 1.0, workspace=workspace),
            "mxfp4_grad_scale": lambda grads: layer.grad_scale(grads, torch.zeros((), dtype=torch.float64), 1.0)}


@pytest.mark.parametrize("name", ["mxfp4_grad_norm", "mxfp4_grad_clip", "mxfp4_grad_scale"])
@pytest.mark.parametrize("given", [False, True])
def test_every_form(recorded, monkeypatch, name, given):  # noqa: F811
    layer, lib = recorded
    a, b = _grad(3, 5), _grad(7)
    seen = []
    real = layer._grads

    def grads_of(grads, out):
        device, items, n = real(grads, out)
        seen.append((n, list(items[2::4])))
        return device, items, n
    monkeypatch.setattr(layer, "_grads", grads_of)
    workspace = _z(8192, dtype=U8) if given else None
    call = _calls(layer, workspace)[name]
    for grads, want in (([a, b], (2, [15, 7])), ((a, b), (2, [15, 7])), ((t for t in (a, b)), (2, [15, 7])), ({0: a, 1: b}.values(), (2, [15, 7])),
                        (a, (1, [15])), (_grad(1).reshape(()), (1, [1])), (_grad(0), (1, [0])), (iter([_grad(0, 3)]), (1, [0]))):
        before = len(lib.calls)
        call(grads)
        assert seen.pop() == want and not seen
        assert [c[0] for c in lib.calls[before:]] == [name]
        if given and name != "mxfp4_grad_scale":
            assert workspace.data_ptr() in lib.calls[-1][1] and 8192 in lib.calls[-1][1]


@pytest.mark.parametrize("name", ["mxfp4_grad_norm", "mxfp4_grad_clip"])
def test_a_workspace_that_cannot_be_used(recorded, name):  # noqa: F811
    layer, lib = recorded
    for workspace in (_z(1, dtype=U8).expand(8192), torch.empty(8192, dtype=U8, device="meta")):
        with pytest.raises(ValueError):
            _calls(layer, workspace)[name]([_grad(3, dtype=F32)])
    assert not lib.calls
