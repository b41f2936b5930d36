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


def scale(grads, out):
    return answer(_lib.load().muon_scale_grads(None, None, tensors(*grads), tensors(*out) if out else None, len(grads), NORM))


FINE, OVERLAP = (MUON_EINVAL, "context NULL"), (MUON_EINVAL, "tensors overlap")


def test_gradients_that_are_only_read_may_overlap():
    """One gradient scaled into two buffers, views of one buffer: every output
    has its own place, so the results do not depend on any order."""
    a, part, b, c = (0x10000, 16, MUON_F32), (0x10010, 4, MUON_F32), (0x20000, 16, MUON_F32), (0x30000, 16, MUON_BF16)
    small = (0x40000, 4, MUON_F32)
    assert scale([a, a], [b, c]) == FINE
    assert scale([a, part], [b, small]) == FINE
    assert scale([part, a], [small, b]) == FINE
    # but nothing that is written
    assert scale([a, a], None) == OVERLAP
    assert scale([a, part], None) == OVERLAP
    assert scale([a, a], [a, b]) == OVERLAP
    assert scale([a, a], [b, a]) == OVERLAP
    assert scale([a, part], [b, part]) == OVERLAP
    assert scale([a, part], [a, small]) == OVERLAP
    assert scale([a, b], [c, (0x30010, 16, MUON_BF16)]) == OVERLAP
    # one that lies inside another and ends first does not hide the overlap of the next
    assert scale([a, part, b], [c, small, (0x1003c, 16, MUON_F32)]) == OVERLAP
    assert scale([a], [(NORM + 8, 16, MUON_F32)]) == OVERLAP
