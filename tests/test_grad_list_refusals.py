"""What lists of gradients are refused, and which are not, without a GPU: the
arguments are checked before the context, with addresses that are never read."""
from newton_schulz_amd import _lib
from newton_schulz_amd._lib import MUON_BF16, MUON_EINVAL, MUON_ESHAPE, MUON_F32, Tensor

NORM = 0x8000


def tensors(*entries):
    return (Tensor * len(entries))(*[Tensor(*e) for e in entries])


def answer(status):
    return status, _lib.load().muon_last_error(None).decode()


def norm(*entries):
    return answer(_lib.load().muon_grad_norm(None, None, tensors(*entries), len(entries), 1.0, 1e-6, NORM))


def test_a_tensor_fits_one_launch():
    """A workgroup of 256 threads for 8192 elements, and one for where the tensor
    starts: fewer than 2^32 threads."""
    most = (1 << 37) - (1 << 14)
    assert (most // 8192 + 1) * 256 < 1 << 32 <= ((most + 8192) // 8192 + 1) * 256
    for dtype in (MUON_BF16, MUON_F32):
        assert norm((0x10000, most, dtype)) == (MUON_EINVAL, "context NULL")
        assert norm((0x10000, most + 1, dtype)) == (MUON_ESHAPE, "tensor numel")
    assert _lib.load().muon_grad_norm_workspace_bytes(tensors((0x10000, most + 1, MUON_BF16)), 1) == 0
    # longer lists take more launches
    assert norm(*[(0x10000 + i * most * 2, most, MUON_BF16) for i in range(9)]) == (MUON_ESHAPE, "too many elements")
    assert norm(*[(0x10000 + i * most * 2, most, MUON_BF16) for i in range(8)]) == (MUON_EINVAL, "context NULL")
