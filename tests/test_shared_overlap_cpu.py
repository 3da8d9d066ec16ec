"""The check of tensors that share memory, against the sets of their bytes."""
import pytest
import torch

from kv_cache_compression_hkv_b200.shared import _overlap


def bytes_of(t):
    at = torch.full((), t.data_ptr(), dtype=torch.int64)
    for n, s in zip(t.shape, t.stride()):
        at = at[..., None] + torch.arange(n) * s * t.element_size()
    return {int(a) + i for a in at.flatten() for i in range(t.element_size())}


def views(base, g):
    """Views [a, b, c, 4] of one buffer: any strides with unit stride in the last dimension."""
    r = lambda lo, hi: int(torch.randint(lo, hi, (), generator=g))  # noqa: E731
    shape = [r(1, 4) for _ in range(3)]
    strides = [r(1, 40) for _ in range(3)] if r(0, 2) else [r(1, 4) * 48, r(1, 4) * 16, r(1, 4) * 4]
    reach = sum((n - 1) * s for n, s in zip(shape, strides)) + 4
    at = r(0, base.numel() - reach + 1)
    return base.as_strided((*shape, 4), (*strides, 1), at)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_overlap_is_that_of_the_bytes(dtype):
    base = torch.empty(1200, dtype=dtype)
    g = torch.Generator().manual_seed(0)
    seen = [0, 0]
    for _ in range(3000):
        x, y = views(base, g), views(base, g)
        want = bool(bytes_of(x) & bytes_of(y))
        assert _overlap(x, y) == want == _overlap(y, x), (x.shape, x.stride(), y.shape, y.stride(), x.storage_offset(), y.storage_offset())
        seen[want] += 1
    assert min(seen) > 300


def test_types_and_ends():
    raw = torch.empty(4096, dtype=torch.uint8)
    f, b = raw.view(torch.float32), raw.view(torch.bfloat16)
    assert not _overlap(f[:8], b[16:32].view(2, 8)) and _overlap(f[:9], b[16:32].view(2, 8))
    wide = b.view(4, 8, 64)
    assert not _overlap(wide[..., :32], wide[..., 32:]) and _overlap(wide[..., :33], wide[..., 32:])
    assert not _overlap(wide[:0], wide) and not _overlap(wide[:2], wide[2:]) and _overlap(wide[:3], wide[2:])
    # large tensors, slices of one: by arithmetic, not by going over the rows
    big = torch.empty(8, 1024, 64, 384, dtype=torch.bfloat16).transpose(1, 2)
    assert not _overlap(big[..., :128], big[..., 128:256]) and _overlap(big[..., :136], big[..., 128:256])
