"""What the classes of the mixer and the optimizer refuse, before any call of the library reaches a GPU:
every operand here lies in host memory."""
import pytest
import torch

from sparse_moe_layer_topk_gb300 import _lib as M
from sparse_moe_layer_topk_gb300 import build as B
from sparse_moe_layer_topk_gb300.linattn import LinearAttention
from sparse_moe_layer_topk_gb300.optim import AdamW

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build_library()
    M.load()


def _mixer(T=8, N=2, Hs=2, r=1, Dk=64, Dv=64, **kw):
    la = LinearAttention(torch.zeros(Hs), T, Dk, Dv, r=r, N=N, **kw)
    return la, [torch.zeros(T, n, w, dtype=BF) for n, w in ((Hs * r, Dk), (Hs, Dk), (Hs, Dv))]


@pytest.mark.parametrize("cu", [
    torch.tensor([0, 3, 8]),                                     # int64, as cumsum makes it of int32 lengths
    torch.tensor([3, 5], dtype=torch.int32).cumsum(0),
    torch.tensor([3, 8], dtype=torch.int32),                     # N entries
    torch.tensor([0, 3, 5, 8], dtype=torch.int32),
    torch.tensor([[0, 3, 8]], dtype=torch.int32),
    torch.tensor([0, 9, 3, 9, 8], dtype=torch.int32)[::2],       # every other entry
    torch.tensor([0.0, 3.0, 8.0])], ids=str)
def test_sequence_bounds_of_another_form(cu):
    la, qkv = _mixer(max_seqlen=8)
    with pytest.raises(ValueError, match="cu_seqlens"):
        la.forward(*qkv, cu)


def test_slots_that_are_not_contiguous():
    la, qkv = _mixer(T=3, N=3)
    state = torch.zeros(6, 2, 64, 64)
    with pytest.raises(ValueError, match="state_idx"):
        la.step(*qkv, state, torch.tensor([0, 9, 1, 9, 2, 9], dtype=torch.int32)[::2])


@pytest.mark.parametrize("stride", [0, 1, 128, 1001, (1 << 32) + 136])
def test_the_stride_of_a_single_token_means_nothing(stride):
    la, _ = _mixer(T=1, N=1)
    x = torch.zeros(128, dtype=BF).as_strided((1, 2, 64), (stride, 64, 1))
    assert la._rows("q", x, 2, 64) == 128


@pytest.mark.parametrize("stride", [1 << 31, (1 << 32) + 128])
def test_tokens_too_far_apart(stride):
    """The library takes the stride as a 32-bit number."""
    la, _ = _mixer(T=2, N=1)
    x = torch.empty_strided((2, 2, 64), (stride, 64, 1), dtype=BF, device="meta")
    with pytest.raises(ValueError, match="apart"):
        la._rows("q", x, 2, 64)


class _OnGpu:
    """A contiguous fp32 tensor of a GPU, as far as a constructor's checks look at one."""
    dtype, is_cuda = torch.float32, True

    def __init__(self, n=10, gpu=0, at=0):
        self.n, self.device, self.at = n, torch.device("cuda", gpu), at

    def data_ptr(self):
        return self.at

    def element_size(self):
        return 4

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True


def test_an_optimizer_of_several_gpus():
    with pytest.raises(ValueError, match="one GPU"):
        AdamW([_OnGpu(), _OnGpu(gpu=1)], [_OnGpu(), _OnGpu(gpu=1)], 1e-3)


@pytest.mark.parametrize("at", [[4096, 4096], [4096, 8192, 4096 + 36], [4096, 4096 + 40, 4096 + 40]], ids=str)
def test_an_optimizer_of_weights_that_share_memory(at):
    with pytest.raises(ValueError, match="share memory"):
        AdamW([_OnGpu(at=a) for a in at], [_OnGpu() for _ in at], 1e-3)


@pytest.mark.parametrize("n", [0, 2])
def test_a_learning_rate_of_no_or_several_values(n):
    with pytest.raises(ValueError, match="one value"):
        AdamW.__new__(AdamW).schedule_on_device(_OnGpu(n))
