"""The workspace that a call takes when it is given none."""
import pytest

torch = pytest.importorskip("torch")


def test_every_call_has_its_own():
    """Two that are held at once, as two threads or a graph and an eager call hold them, share no
    byte, whatever their sizes."""
    import bit_weight_only_offline_amd as Q
    held = [Q.workspace("cpu", n) for n in (1000, 1000, 10, 100000, 0)]
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel()) for t in held)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    assert all(t.dtype == torch.uint8 and t.is_contiguous() for t in held)
    assert [t.numel() for t in held] == [1000, 1000, 256, 100000, 256]
