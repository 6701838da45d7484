"""Numbers that no integer argument holds, and what is no number, are refused with the binding's own
error before anything is launched.  A float over fp32's range is infinity there: the update refuses
that, a product's scale may be.  Host tensors stand in for device ones."""
import pytest
import torch


@pytest.fixture(scope="module")
def eg():
    import hashed_gram_memory_gb300 as eg
    return eg


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)


def zeros(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


def bf(*shape):
    return zeros(*shape, dtype=torch.bfloat16)


REFUSED = {
    "scale of text": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), scale="one", out=zeros(4, 5), stream=1),
    "activation over 32 bits": lambda e: e.engram_matmul(bf(4, 8), bf(5, 8), activation=2 ** 40, out=zeros(4, 5), stream=1),
    "update's scale of text": lambda e: e.engram_orthogonalise(zeros(8, 8), out=bf(8, 8), scale="one", stream=1,
                                                               workspace=zeros(1 << 16, dtype=torch.uint8)),
    "steps in halves": lambda e: e.engram_orthogonalise(zeros(8, 8), out=bf(8, 8), steps=2.5, stream=1,
                                                        workspace=zeros(1 << 16, dtype=torch.uint8)),
    "steps over 32 bits": lambda e: e.engram_orthogonalise(zeros(8, 8), out=bf(8, 8), steps=2 ** 32 + 5, stream=1,
                                                           workspace=zeros(1 << 16, dtype=torch.uint8)),
    "beta over fp32": lambda e: e.engram_orthogonalise(zeros(8, 8), out=bf(8, 8), beta=1e60, stream=1,
                                                       workspace=zeros(1 << 16, dtype=torch.uint8)),
}


@pytest.mark.parametrize("what", REFUSED)
def test_numbers_out_of_range(eg, what):
    with pytest.raises(eg.EngramError) as e:
        REFUSED[what](eg)
    assert e.value.code == eg.ERR_INVALID_ARG, str(e.value)
