"""The calls' workspace comes from torch's allocator, by whichever of its functions this torch has: no GPU."""
from types import SimpleNamespace

import pytest

from skinny_bf16_split_gb300 import _binding as b


def fake(private):
    """A torch of one device whose allocator keeps a log."""
    log = []
    alloc = lambda size, stream: log.append(("alloc", size, stream)) or 4096  # noqa: E731
    free = lambda address: log.append(("free", address))  # noqa: E731
    C = SimpleNamespace(_cuda_getDevice=lambda: 0, _cuda_getCurrentRawStream=lambda index: 77)
    cuda = SimpleNamespace()
    if private:
        C._cuda_cudaCachingAllocator_raw_alloc, C._cuda_cudaCachingAllocator_raw_delete = alloc, free
    else:
        cuda.caching_allocator_alloc = lambda size, device=None, stream=None: alloc(size, stream)
        cuda.caching_allocator_delete = free
    return SimpleNamespace(_C=C, cuda=cuda), log


@pytest.mark.parametrize("private", [True, False])
@pytest.mark.parametrize("stream,raw", [(None, 77), (5, 5)])
@pytest.mark.parametrize("refused", [True, False])
def test_workspace(monkeypatch, private, stream, raw, refused):
    torch, log = fake(private)
    monkeypatch.setattr(b, "_torch", lambda: torch)
    b._allocator.cache_clear()
    args = b.dep_attention_args_t()

    def call(args, stream):
        log.append(("call", args.workspace, args.workspace_bytes, stream))
        if refused:
            raise b.DepError(1, "call")

    try:
        if refused:
            with pytest.raises(b.DepError):
                b._on_with_workspace(0, call, args, 1000, stream)
        else:
            b._on_with_workspace(0, call, args, 1000, stream)
    finally:
        b._allocator.cache_clear()
    assert log == [("alloc", 1000, raw), ("call", 4096, 1000, raw), ("free", 4096)]
