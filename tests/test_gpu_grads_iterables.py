"""Gradients as any iterable: tensors that only the call itself holds stay alive
until it has been enqueued, and its scratch is not their memory."""
import pytest
import torch

from lossless_bf16_tensor_gb300.grads import clip_grads, grad_norm
from test_gpu_grads import check_clipped, check_norm, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# sizes whose blocks are those of the norm (512 bytes) and of the scratch (5 KB), among others
SIZES = [1, 100, 128, 1224, 1225, 1280, 2448, 2560, 5000, 70_000] * 3


class Made:
    """A sequence that makes its tensors when they are asked for."""

    def __init__(self, gs):
        self.gs = gs

    def __len__(self):
        return len(self.gs)

    def __getitem__(self, i):
        return self.gs[i] * 1


@pytest.mark.parametrize("dtypes", [[BF], [F32], [BF, F32]], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("count", [1, 4, len(SIZES)])
def test_tensors_made_on_the_way(count, dtypes):
    gs = make(SIZES[-count:], dtypes, seed=count, scale=1.0)
    for _ in range(3):
        check_norm(grad_norm(g * 1 for g in gs), gs)
        check_norm(grad_norm(Made(gs)), gs)
        check_norm(grad_norm(tuple(gs)), gs)
        out = [torch.zeros_like(g) for g in gs]
        check_clipped(clip_grads((g * 1 for g in gs), 0.5, out=(o.view(-1) for o in out)), out, gs, 0.5)
        made = [g.clone() for g in gs]
        check_clipped(clip_grads((g.view(-1) for g in made), 0.5), made, gs, 0.5)


def test_what_is_no_iterable_of_tensors():
    for bad in (None, 3, [None], (torch.zeros(2, device="cuda"), "x")):
        with pytest.raises((TypeError, ValueError)):
            grad_norm(bad)

    def fails():
        yield torch.zeros(2, device="cuda")
        raise KeyError("gone")
    with pytest.raises(KeyError):
        grad_norm(fails())
    with pytest.raises(ValueError):
        clip_grads([torch.zeros(2, device="cuda")], 1.0, out=iter(()))
